"""The block operators at the largest row counts that their argument checks admit, with the tolerances derived in
test_block_gpu."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpNorm  # noqa: E402
from tests.test_block_gpu import (EPS, check_linear_backward, check_linear_forward, check_norm_backward,  # noqa: E402
                                  check_norm_forward, norm_case, norm_ref)

MOST = 1 << 24


@pytest.mark.parametrize("rows,H", [(70001, 5), (MOST, 2), (MOST, 7)])
def test_norm_of_short_rows(rows, H):
    """Rows of fewer than 8 elements, more of them than workgroups."""
    check_norm_forward(rows, H, "f16")
    check_norm_backward(rows, H, "bf16")


@pytest.mark.parametrize("H", [8, 12])
def test_norm_of_most_rows(H):
    check_norm_forward(MOST, H, "bf16")
    check_norm_backward(MOST, H, "f16")


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_linear_layer_of_most_rows(act):
    check_linear_forward(MOST, 8, 16, act, "f16")
    check_linear_backward(MOST, 16, 8, act, "f16")


@pytest.mark.parametrize("H", [5, 264, 333, 20000])
def test_norm_of_one_token_of_each_long_sequence(H):
    """Rows further apart than 2^24 elements, as the last tokens of a batch of long sequences are."""
    rows, ld = 20, (1 << 25) + 24
    x, w, b, dy, dres = norm_case(rows, H, "bf16", 5)
    _, mean, rstd, _ = norm_ref(x, w, b)
    base = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda").view(rows, ld)
    at = lambda k: base[:, k * 32768:k * 32768 + H]  # noqa: E731
    with MlpNorm(H, "bf16", EPS) as layer:
        outs = []
        for far in (False, True):
            place = (lambda k, t: at(k).copy_(t)) if far else (lambda k, t: t.clone())
            y, dx = place(0, torch.zeros_like(x)), place(1, torch.zeros_like(x))
            dw, db = torch.zeros_like(w), torch.zeros_like(b)
            layer.forward(place(2, x), w, b, y)
            layer.backward(place(3, dy), place(2, x), w, mean.float(), rstd.float(), dx, dw, db, dres=place(4, dres))
            outs.append((y, dx, dw, db))
    assert all(torch.equal(p, q) for p, q in zip(*outs)) and bool(outs[0][0].isfinite().all())
