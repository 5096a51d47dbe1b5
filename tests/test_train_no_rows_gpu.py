"""Calls of the cross entropy whose rows are all left out, on tall tiles and in pieces: every output is zero, and what a
canary around it held is still there."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLoss  # noqa: E402
from consumer_gemm_chain_amd import mlp_train as mt  # noqa: E402

TALL = 4        # the tile configuration of 160 to 256 rows
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def outputs(rows, H, V, dtype):
    """loss, lse, dx and dw full of sevens, each the front of a buffer with as many more behind it."""
    base = [torch.full((2 * n, *more), 7.0, dtype=t, device="cuda")
            for n, more, t in ((rows, (), torch.float32), (rows, (), torch.float32), (rows, (H,), DT[dtype]), (V, (H,), DT[dtype]))]
    return [b[:len(b) // 2] for b in base], [b[len(b) // 2:] for b in base]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H,V,most", [(257, 136, 1500, None), (512, 136, 1500, None), (700, 64, 300, None),
                                           (600, 64, 1001, 1 << 20)])
def test_no_row_counts_on_tall_tiles(rows, H, V, most, dtype):
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.full((rows, H), float("nan"), device="cuda").to(DT[dtype])
    w = torch.randn(V, H, generator=g, device="cuda").to(DT[dtype])
    target = torch.full((rows,), -1, device="cuda")
    with MlpLoss(most or rows, H, V, dtype) as layer:
        for product in (0, 1):
            mt.mlp_loss_debug_set_plan(layer.h, product, TALL, 0)
        for wanted in ("xw", "x", "w"):
            (loss, lse, dx, dw), behind = outputs(rows, H, V, dtype)
            layer.forward(x, w, target, loss, lse)
            layer.backward(x, w, target, lse, dx=dx if "x" in wanted else None, dw=dw if "w" in wanted else None)
            torch.cuda.synchronize()
            assert (loss == 0).all() and (lse == 0).all()
            assert (dx == (0 if "x" in wanted else 7)).all() and (dw == (0 if "w" in wanted else 7)).all()
            assert all((t == 7).all() for t in behind)
        # a target beyond the vocabulary counts as little
        (loss, lse, dx, dw), behind = outputs(rows, H, V, dtype)
        target.fill_(V)
        layer.forward(x, w, target, loss, lse)
        layer.backward(x, w, target, lse, dx=dx, dw=dw)
        torch.cuda.synchronize()
        assert loss.isnan().all() and lse.isnan().all() and (dx == 0).all() and (dw == 0).all()
        assert all((t == 7).all() for t in behind)
