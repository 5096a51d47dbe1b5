"""The block operators' paths that only long, wide or far-apart operands reach: loops that take a second step,
ragged rows wider than a wave holds, and rows further apart than 32-bit offsets, with the tolerances derived in
test_block_gpu."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLinear  # noqa: E402
from consumer_gemm_chain_amd import mlp_block as mb  # noqa: E402
from tests.test_block_gpu import check_norm_backward, check_norm_forward, linear_case  # noqa: E402


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H", [(8195, 264), (8193, 1000), (8200, 2048), (2049, 4096), (2100, 8192), (2060, 8187),
                                    (2100, 12281), (2049, 16384), (5, 2049), (5, 4095), (3, 12283), (5, 16383)])
def test_norm_forward_of_many_rows_and_ragged_widths(rows, H, dtype):
    """2048 workgroups of one or four rows: more rows than one step of them, the last step partly filled; and every
    register-held width that ends inside a chunk."""
    check_norm_forward(rows, H, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H", [(9001, 500), (3001, 2041), (1101, 4095), (700, 8191), (600, 9001), (600, 12288),
                                    (530, 12295), (520, 16384), (3, 9001), (3, 16383)])
def test_norm_backward_of_many_rows_and_ragged_widths(rows, H, dtype):
    """256 workgroups that take three and more steps, with the next row's loads in flight and the columns' sums carried."""
    check_norm_backward(rows, H, dtype)


@pytest.mark.parametrize("rows,H", [(700, 8191), (600, 9001), (530, 12295)])
def test_norm_backward_of_many_rows_in_place_and_without_residual(rows, H):
    check_norm_backward(rows, H, "bf16", in_place=True)
    check_norm_backward(rows, H, "f16", dres=False, weight=False)
    check_norm_backward(rows, H, "f16", pad=5)


@pytest.mark.parametrize("forced", [False, True])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_every_operand_past_32_bits(act, forced):
    """Every operand and output of the linear layer in rows 2^23 elements apart, whose last rows lie past 2^32 bytes,
    by the planner's choice and with the reductions split: the bits of packed operands."""
    rows, K, N, ld = 300, 520, 264, 1 << 23
    c = linear_case(rows, K, N, act, "bf16", 6)
    gN = c["gN"]
    base = torch.empty(K * ld, dtype=torch.bfloat16, device="cuda").view(K, ld)
    at = [0]

    def far(t):
        """A copy of `t` in columns of its own of the wide buffer."""
        view = base[: t.shape[0], at[0]:at[0] + t.shape[1]]
        at[0] += 1024
        view.copy_(t)
        return view

    x, w, res, dy = c["x"], c["w"], c["res"], c["dy"]
    z = c["z"] if act != "none" else None
    outs = []
    with MlpLinear(rows, K, N, act, "bf16") as layer:
        if forced:
            for op in range(3):
                mb.mlp_linear_debug_set_plan(layer.h, op, 2, 3)
        for place in (lambda t: t.clone(), far):
            new = lambda *shape: place(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))  # noqa: E731
            y, h, dx, dw = new(rows, N), new(rows, gN), new(rows, K), new(K, gN)
            db = torch.empty_like(c["bias"])
            layer.forward(place(x), place(w), y, bias=c["bias"], residual=place(res), z=h)
            layer.backward(place(dy), place(x), place(w), dx=dx, dw=dw, db=db, z=place(z) if z is not None else None)
            outs.append([y, h, dx, dw, db])
        torch.cuda.synchronize()
    assert at[0] <= ld
    assert all(bool(t.float().abs().sum() > 0) for t in outs[0])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
