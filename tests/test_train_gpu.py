"""Cross entropy, gradient norm and AdamW on the GPU, through the binding, against the definitions in 64 bits.

Tolerances.  u is the storage type's unit roundoff; an output is rounded once: u |ref|, plus fp16's half subnormal
step.  An fp32 sum of n terms on the matrix cores errs by at most (n/32 + 64) 2^-23 sum|terms|.  Elementwise fp32
arithmetic (a handful of operations, hardware 2^x, root and reciprocal) errs by 2^-20 of its largest term.  dz is
rounded to the storage type (u each, in fp16 at least 2^-25 of the unit): independent errors of at most u |dz W|, for
which eight times their root of the sum of squares is allowed.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW, MlpChainError, MlpGradNorm, MlpLoss  # noqa: E402
from consumer_gemm_chain_amd import mlp_train as mt  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
E32 = 2.0 ** -23


def gen(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return g, lambda *shape: torch.randn(shape, generator=g, device="cuda")


def padded(t, pad, rows=0):
    """`t` as a view with `pad` more elements per row and `rows` more rows, which hold NaN."""
    base = torch.full((t.shape[0] + rows, t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = base[:t.shape[0], :t.shape[1]]
    view.copy_(t)
    return view


def canary(rows, cols, dtype, pad=0):
    """An output filled with a canary, and a check that its padding still holds it."""
    base = torch.full((rows + 2, cols + pad), 77.0, dtype=DT[dtype], device="cuda")
    return base[:rows, :cols], lambda: bool((base[:, cols:] == 77.0).all() and (base[rows:] == 77.0).all())


def close(got, ref, tol, what):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(got[bad][0]), float(ref[bad][0]),
                           float(torch.as_tensor(tol).expand_as(ref)[bad][0]))


# ------------------------------------------------------------------------ loss

def loss_case(rows, H, V, dtype, seed, left_out="some", spread=3.0):
    g, n = gen(seed)
    dt = DT[dtype]
    x, w = n(rows, H).to(dt), (n(V, H) * (spread / math.sqrt(H))).to(dt)
    target = torch.randint(V, (rows,), generator=g, device="cuda")
    if left_out == "some":
        target = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.3, -100, target)
    elif left_out == "all":
        target = torch.full_like(target, -1)
    return x, w, target


def loss_ref(x, w, target):
    """z, lse, loss, and a bound of the error of each z."""
    x, w = x.double(), w.double()
    z = x @ w.t().contiguous()
    ez = (x.shape[1] / 32 + 64) * E32 * (x.abs() @ w.t().abs().contiguous())
    lse = torch.logsumexp(z, 1)
    rows = torch.arange(len(target), device=x.device)
    at = z[rows, target.clamp(min=0)]
    counted = target >= 0
    return z, torch.where(counted, lse, 0.0), torch.where(counted, lse - at, 0.0), ez


def check_loss_forward(rows, H, V, dtype, left_out="some", pad=0, seed=1, plan=None, spread=3.0):
    x, w, target = loss_case(rows, H, V, dtype, seed, left_out, spread)
    loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    with MlpLoss(rows, H, V, dtype, grad=False) as layer:
        if plan is not None:
            mt.mlp_loss_debug_set_plan(layer.h, 0, plan, 0)
        layer.forward(padded(x, pad, 1), padded(w, pad, 1), target, loss, lse)
        torch.cuda.synchronize()
    z, rlse, rloss, ez = loss_ref(x, w, target)
    tol = ez.amax(1) + 2.0 ** -20 + (V / 4096 + 64) * E32 + 2 * E32 * rlse.abs()
    close(lse, rlse, tol, "lse")
    close(loss, rloss, 2 * tol + 2 * E32 * rloss.abs(), "loss")
    assert (loss[target < 0] == 0).all() and (lse[target < 0] == 0).all()


SIZES = [(1, 8, 1), (1, 8, 2), (2, 16, 3), (1, 64, 7), (3, 72, 8), (1, 512, 1000), (5, 136, 129), (16, 512, 255), (17, 64, 256),
         (48, 200, 257), (64, 1024, 1000), (65, 64, 513), (100, 520, 2001), (129, 512, 700), (200, 64, 5003), (256, 128, 1024),
         (257, 328, 999), (300, 1096, 3001), (600, 64, 40001), (1000, 512, 777)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H,V", SIZES)
def test_loss_forward(rows, H, V, dtype):
    check_loss_forward(rows, H, V, dtype)


@pytest.mark.parametrize("left_out", ["none", "all"])
@pytest.mark.parametrize("rows,H,V", [(1, 64, 100), (70, 72, 300), (600, 136, 513)])
def test_loss_forward_rows_left_out(rows, H, V, left_out):
    check_loss_forward(rows, H, V, "bf16", left_out)


@pytest.mark.parametrize("rows,H,V", [(1, 64, 100), (70, 72, 300), (600, 136, 513)])
def test_loss_forward_strides(rows, H, V):
    check_loss_forward(rows, H, V, "f16", pad=8)
    check_loss_forward(rows, H, V, "f16", pad=64)


@pytest.mark.parametrize("spread", [0.0, 0.1, 30.0])
def test_loss_forward_of_flat_and_peaked_rows(spread):
    """Equal logits (lse = log V) to a spread where a single word has nearly all of the probability."""
    check_loss_forward(40, 128, 1003, "bf16", spread=spread)
    check_loss_forward(300, 128, 1003, "bf16", spread=spread)


def check_loss_backward(rows, H, V, dtype, left_out="some", pad=0, seed=2, dloss="mean", dlse=False, outputs="xw", plan=None,
                        split=0, most=None):
    x, w, target = loss_case(rows, H, V, dtype, seed, left_out)
    _, n = gen(seed + 100)
    z, lse, _, ez = loss_ref(x, w, target)
    lse = lse.float()
    counted = target >= 0
    if dloss == "mean":
        d = torch.full((rows,), 1.0 / max(1, int(counted.sum())), device="cuda")
    else:
        d = torch.ones(rows, device="cuda") if dloss is None else n(rows)
    dl = 0.1 * n(rows) if dlse else None
    if dtype == "f16":
        d, dl = d * 64, dl * 64 if dlse else None
        if dloss is None:
            d = torch.ones_like(d)
    # values that belong to rows left out do not matter
    garbage = torch.where(counted, d, math.nan)
    dx, okx = canary(rows, H, dtype, pad)
    dw, okw = canary(V, H, dtype, pad)
    with MlpLoss(most or rows, H, V, dtype) as layer:
        if plan is not None:
            mt.mlp_loss_debug_set_plan(layer.h, 1, plan, split)
            mt.mlp_loss_debug_set_plan(layer.h, 0, plan, 0)
        layer.backward(padded(x, pad, 1), padded(w, pad, 1), target, lse, None if dloss is None else garbage, dl,
                       dx=dx if "x" in outputs else None, dw=dw if "w" in outputs else None)
        torch.cuda.synchronize()
    a = torch.where(counted, d.double() + (dl.double() if dlse else 0.0), 0.0)
    b = torch.where(counted, d.double(), 0.0)
    p = torch.exp(z - lse.double()[:, None])
    dz = a[:, None] * p
    hot = torch.zeros_like(dz)
    hot[torch.arange(rows, device="cuda"), target.clamp(min=0)] = 1.0
    dz = dz - b[:, None] * hot
    unit = float(torch.maximum(a.abs(), b.abs()).max()) * (2.0 ** -14 if dtype == "f16" else 1.0)
    each = U[dtype] * dz.abs() + TINY[dtype] * unit                     # rounding of dz
    soft = a.abs()[:, None] * p * (ez + 2.0 ** -18) + 2.0 ** -20 * (dz.abs() + b.abs()[:, None] * hot)
    w64, x64 = w.double(), x.double()
    each, soft = each * counted[:, None], soft * counted[:, None]
    t = lambda m: m.t().contiguous()  # noqa: E731
    if "x" in outputs:
        ref = dz @ w64
        tol = U[dtype] * ref.abs() + TINY[dtype] + 8 * torch.sqrt(each.square() @ w64.square())
        tol += soft @ w64.abs() + (V / 32 + 64) * E32 * (dz.abs() @ w64.abs())
        close(dx, ref, tol, "dx")
        assert (dx[~counted] == 0).all()
    if "w" in outputs:
        ref = t(dz) @ x64
        tol = U[dtype] * ref.abs() + TINY[dtype] + 8 * torch.sqrt(t(each.square()) @ x64.square())
        tol += t(soft) @ x64.abs() + (rows / 32 + 64) * E32 * (t(dz.abs()) @ x64.abs())
        close(dw, ref, tol, "dw")
    assert okx() and okw(), "padding was written"
    for out, name in ((dx, "x"), (dw, "w")):
        assert name in outputs or (out == 77.0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H,V", SIZES)
def test_loss_backward(rows, H, V, dtype):
    check_loss_backward(rows, H, V, dtype)


@pytest.mark.parametrize("left_out", ["none", "all"])
@pytest.mark.parametrize("rows,H,V", [(1, 64, 100), (70, 72, 300), (600, 136, 513)])
def test_loss_backward_rows_left_out(rows, H, V, left_out):
    check_loss_backward(rows, H, V, "bf16", left_out)


@pytest.mark.parametrize("outputs", ["x", "w"])
@pytest.mark.parametrize("rows,H,V", [(3, 64, 1), (70, 72, 300), (600, 136, 513)])
def test_loss_backward_single_outputs(rows, H, V, outputs):
    check_loss_backward(rows, H, V, "f16", outputs=outputs)
    check_loss_backward(rows, H, V, "bf16", outputs=outputs, pad=16)


@pytest.mark.parametrize("dloss,dlse", [(None, False), ("any", False), ("any", True), ("mean", True)])
@pytest.mark.parametrize("rows,H,V", [(9, 64, 100), (300, 72, 777)])
def test_loss_backward_upstream_gradients(rows, H, V, dloss, dlse):
    check_loss_backward(rows, H, V, "f16", dloss=dloss, dlse=dlse)
    check_loss_backward(rows, H, V, "bf16", dloss=dloss, dlse=dlse)
