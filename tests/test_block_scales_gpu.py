"""Layer norm of rows whose spread is far from one (bf16, whose range is fp32's), without eps."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpNorm  # noqa: E402
from tests.test_block_gpu import gen  # noqa: E402

U = 2.0 ** -8


@pytest.mark.parametrize("spread", [1e15, 1e-15, 3e-20, 1e-20])
@pytest.mark.parametrize("rows,H", [(9, 5), (5, 333), (60, 512), (5, 8192), (5, 9001), (5, 16384), (5, 20000)])
def test_norm_of_small_and_large_rows(rows, H, spread):
    """rstd from 1e-15 to 1e20; the gradient's terms are of rstd's size, not of its square.  Every output is rounded
    once, by at most u of itself, and the fp32 arithmetic (variances down to 1e-40, of 16 bits) errs by far less:
    relative 2-norms within u."""
    n = gen(81)
    x = (spread * n(rows, H)).bfloat16()
    w, b, dy = (1 + 0.1 * n(H)).bfloat16(), (0.1 * n(H)).bfloat16(), (0.1 * n(rows, H)).bfloat16()
    y, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    with MlpNorm(H, "bf16", 0.0) as layer:
        layer.forward(x, w, b, y, mean, rstd)
        layer.backward(dy, x, w, mean, rstd, dx, dw, db)
        torch.cuda.synchronize()
    xd, wd, dyd = x.double(), w.double(), dy.double()
    c = xd - xd.mean(1, keepdim=True)
    rs = 1 / torch.sqrt((c * c).mean(1, keepdim=True))
    xhat, g = c * rs, dyd * wd
    ref = {"y": (y, xhat * wd + b.double()), "rstd": (rstd, rs[:, 0]), "dweight": (dw, (dyd * xhat).sum(0)), "dbias": (db, dyd.sum(0)),
           "dx": (dx, rs * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)))}
    for name, (got, want) in ref.items():
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= U, (name, rel)
