"""The cross entropy at the ends of what its header allows: the most words, the longest rows, the largest row strides."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLoss  # noqa: E402
from tests.test_train_gpu import DT, check_loss_backward, check_loss_forward, loss_case  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H,V", [(3, 8, (1 << 22) - 1), (300, 8, 500001), (3, (1 << 22) - 8, 9), (70, 262152, 33)])
def test_wide_and_long(rows, H, V, dtype):
    check_loss_forward(rows, H, V, dtype)
    check_loss_backward(rows, H, V, dtype)


def far_apart(t, ld):
    """`t` as a view whose rows are `ld` elements apart."""
    base = torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device=t.device)
    view = torch.as_strided(base, t.shape, (ld, 1))
    view.copy_(t)
    return view


@pytest.mark.parametrize("left_out", ["none", "some"])
@pytest.mark.parametrize("rows", [2, 63, 64, 100, 200, 256, 257, 400])
def test_the_largest_row_strides(rows, left_out):
    """Operands and outputs as far apart as they may be: the bits of the call on neighbouring rows."""
    H, V, dtype = 136, 70, "bf16"
    x, w, target = loss_case(rows, H, V, dtype, 3, left_out)
    if left_out == "some":
        target[0], target[1] = -1, 3
    most = max(1 << 23, ((1 << 31) - (1 << 24)) // rows) // 8 * 8
    assert most == 1 << 23 or rows < 256
    results = []
    with MlpLoss(rows, H, V, dtype) as layer:
        for far in (False, True):
            loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
            place = far_apart if far else lambda t, ld: t.clone()
            xs, ws = place(x, most), place(w, 1 << 23)
            dx = place(torch.full_like(x, 7.0), (1 << 33) // rows // 8 * 8)
            dw = place(torch.full_like(w, 7.0), 1 << 27)
            layer.forward(xs, ws, target, loss, lse)
            layer.backward(xs, ws, target, lse, dx=dx, dw=dw)
            torch.cuda.synchronize()
            results.append([t.clone() for t in (loss, lse, dx.contiguous(), dw.contiguous())])
            del xs, ws, dx, dw
            torch.cuda.empty_cache()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert results[0][2].isfinite().all() and results[0][3].any() and results[0][2].dtype == DT[dtype]
