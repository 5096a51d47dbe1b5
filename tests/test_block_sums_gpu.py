"""Long fp32 sums of the norm: their chains stay short."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpNorm  # noqa: E402
from tests.test_block_gpu import DT, gen  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H", [20001, 1 << 20, 1 << 22])
@pytest.mark.parametrize("offset", [0.0, 1000.0])
def test_rstd_of_long_rows(H, offset, dtype):
    """A sum of H positive terms in chains of at most 64, then one per 16384, then 10 across the workgroup: relative
    error at most (64 + H / 16384 + 10) 2^-24, half of it in rstd, and a few roundings of single operations.  The
    variance is the one around the kernel's own mean, whose error is bounded by the same chain."""
    x = (offset + gen(91)(3, H)).to(DT[dtype])
    y = torch.empty_like(x)
    mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    with MlpNorm(H, dtype, 1e-5, grad=False) as layer:
        layer.forward(x, None, None, y, mean, rstd)
        torch.cuda.synchronize()
    chain = (64 + H / 16384 + 10) * 2.0 ** -24
    xd = x.double()
    assert bool(((mean.double() - xd.mean(1)).abs() <= (chain + 2.0 ** -23) * xd.abs().mean(1)).all())
    d = xd - mean.double()[:, None]
    want = 1 / torch.sqrt((d * d).mean(1) + 1e-5)
    assert float(((rstd.double() - want) / want).abs().max()) <= chain / 2 + 4 * 2.0 ** -23


@pytest.mark.parametrize("rows,H", [(1 << 20, 3), (1 << 22, 2)])
def test_column_sums_of_short_rows(rows, H):
    """The gradients of weight and bias over many rows of all-positive terms: chains of 64, then of the group's."""
    n = gen(92)
    x, dy = n(rows, H).half(), (1 + n(rows, H).abs()).bfloat16().half()
    w = torch.ones(H, dtype=torch.float16, device="cuda")
    mean, rstd = torch.full((rows,), -8.0, device="cuda"), torch.full((rows,), 2.0 ** -12, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    scale = 2.0 ** -8       # (fp16 holds the sums)
    with MlpNorm(H, "f16", 1e-5) as layer:
        layer.backward((dy.float() * scale).half(), x, w, mean, rstd, dx, dw, db)
        torch.cuda.synchronize()
    d = (dy.float() * scale).half().double()
    xhat = (x.double() + 8) * 2.0 ** -12
    chain = (64 + rows / 64 / 64 + 64 + 10) * 2.0 ** -24
    for got, want in ((dw, (d * xhat).sum(0)), (db, d.sum(0))):
        assert bool(((got.double() - want).abs() <= (2.0 ** -11 + chain + 4 * 2.0 ** -23) * want.abs()).all())
