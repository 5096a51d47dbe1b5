"""The linear layer's planner on the host: tiles cover the product, parts are
not empty, only the last round is split, and the workspace stays bounded."""
import itertools

import pytest

from consumer_gemm_chain_amd import mlp_block as mb
from consumer_gemm_chain_amd import mlp_chain as mc

ACT = {"none": 0, "gelu_tanh": 1, "swiglu": 2}
ROWS = (1, 2, 7, 16, 17, 64, 65, 100, 128, 129, 300, 512, 515, 769, 1000, 2048, 2049, 5000, 8192)
SIZES = ((8, 8), (64, 64), (72, 40), (512, 2048), (2048, 512), (3584, 8192), (6144, 12288), (8192, 2752), (12288, 6144))


@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("cus", [8, 64, 256, 304])
def test_plans_are_sound(K, N, cus):
    for rows, act, op in itertools.product(ROWS, ("none", "swiglu"), range(5)):
        p = mb.mlp_linear_plan(rows, K, N, ACT[act], op, cus)
        gN = N * (2 if act == "swiglu" else 1)
        m, n, k = ((rows, gN, K), (rows, K, gN), (K, gN, rows), (rows, K, gN), (K, gN, rows))[op]
        what = (rows, K, N, act, op, cus, p)
        assert p["Mt"] == -(-m // p["BM"]) and p["Nt"] == -(-n // p["BN"]), what
        tiles, slabs = p["Mt"] * p["Nt"], k // 64
        assert 1 <= p["S"] <= 32, what
        if p["S"] == 1:
            assert p["part_bytes"] == 0, what
            continue
        # every part has slabs, together they are all of them
        assert (p["S"] - 1) * p["ksp"] < slabs <= p["S"] * p["ksp"], what
        # whole rounds of the chip are never split, and the rest makes at most one
        assert p["direct"] == tiles - tiles % cus and p["direct"] < tiles, what
        assert (tiles - p["direct"]) * p["S"] <= cus, what
        assert p["part_bytes"] == (tiles - p["direct"]) * p["S"] * p["BM"] * p["BN"] * 4 <= cus * 256 * 1024, what
        if op not in (2, 4):
            assert p["BM"] <= max(64, 2 * rows), what


def test_plans_follow_the_rows():
    """A single token streams weights over most of the chip; large batches take the largest tiles unsplit."""
    one = mb.mlp_linear_plan(1, 12288, 6144, 0, 0, 256)
    assert one["BM"] <= 64 and one["S"] > 1 and 192 <= one["Mt"] * one["Nt"] * one["S"] <= 256
    big = mb.mlp_linear_plan(8192, 12288, 6144, 0, 0, 256)
    assert big["BM"] == 256
    assert mb.mlp_linear_plan(8, 64, 64, 0, 0, 256)["S"] == 1


@pytest.mark.parametrize("K,N", SIZES)
def test_both_products_in_one_launch(K, N):
    """One configuration for both, at most one of them split."""
    for rows, act in itertools.product(ROWS, ("none", "swiglu")):
        dx, dw = (mb.mlp_linear_plan(rows, K, N, ACT[act], op, 256) for op in (3, 4))
        assert dx["config"] == dw["config"] and min(dx["S"], dw["S"]) == 1, (rows, act, dx, dw)


@pytest.mark.parametrize("args,needle", [
    ((0, 64, 64, 0, 0, 256), "rows"),
    ((4, 60, 64, 0, 0, 256), "multiples of 8"),
    ((4, 64, 64, 5, 0, 256), "activation"),
    ((4, 64, 64, 0, 5, 256), "pass"),
    ((4, 64, 64, 0, -1, 256), "pass"),
    ((4, 64, 64, 0, 0, 4), "cus"),
])
def test_plan_refuses(args, needle):
    with pytest.raises(mc.MlpChainError, match=needle):
        mb.mlp_linear_plan(*args)


def test_plan_needs_an_array():
    assert mb._library().mlp_linear_plan(4, 64, 64, 0, 0, 256, None, 9) == mc.MLP_EINVAL
    assert mb._library().mlp_linear_debug_set_plan(None, 0, 0, 1) == mc.MLP_EINVAL
