"""The block operators at the largest row counts that their argument checks admit, with the tolerances derived in
test_block_gpu."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpChainError, MlpLinear, MlpNorm  # noqa: E402
from consumer_gemm_chain_amd import mlp_block as mb  # noqa: E402
from tests.test_block_gpu import (EPS, check_linear_backward, check_linear_forward, check_norm_backward,  # noqa: E402
                                  check_norm_forward, linear_case, norm_case, norm_ref)

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


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows", [1, 20, 70])
def test_linear_layer_of_one_token_of_each_long_sequence(rows, act):
    """Every operand but the weights in rows further apart than 2^23 elements; strides that 32-bit offsets within a
    tile would not reach are refused."""
    K, N = 328, 264
    ld = (1 << 24) + 24
    c = linear_case(rows, K, N, act, "f16", 5)
    gN, w, bias = c["gN"], c["w"], c["bias"]
    base = torch.empty(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)
    at = lambda k, n: base[:, k * 4096:k * 4096 + n]  # noqa: E731
    z = c["z"] if act != "none" else None
    outs = []
    with MlpLinear(300, K, N, act, "f16") as layer:
        for far in (False, True):
            place = (lambda k, t: at(k, t.shape[1]).copy_(t)) if far else (lambda k, t: t.clone())
            y, h, dx = (place(k, torch.zeros(rows, n, device="cuda").half()) for k, n in enumerate((N, gN, K)))
            dw, db = torch.zeros_like(w), torch.zeros_like(bias)
            layer.forward(place(3, c["x"]), w, y, bias=bias, residual=place(4, c["res"]), z=h)
            layer.backward(place(5, c["dy"]), place(3, c["x"]), w, dx=dx, dw=dw, db=db, z=place(6, z) if z is not None else None)
            outs.append((y, h, dx, dw, db))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(*outs)) and bool(outs[0][0].isfinite().all())
        p = base.data_ptr()
        with pytest.raises(MlpChainError, match="row stride of x"):
            mb.mlp_linear_forward(layer.h, 300, p, ld, w.data_ptr(), gN, None, None, 0, p, N, None, 0, None)
