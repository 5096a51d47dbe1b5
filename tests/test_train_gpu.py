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


@pytest.mark.parametrize("rows", [5, 300])
def test_the_loss_of_a_confident_row_does_not_suffer_from_the_size_of_its_logits(rows):
    """Logits are exact here: 1000 at the target, 992 elsewhere, so loss = log(1 + 199 e^-8), of which fp32 sums near one
    (at most 32 roundings of 2^-24) and 2^x (2^-20 of the other terms' sum) leave 2e-6; half a step of lse is 3e-5."""
    at = torch.arange(rows, device="cuda") % 8
    x = torch.nn.functional.one_hot(at, 8).bfloat16()
    w = torch.full((200, 8), 992.0, device="cuda").bfloat16()
    w[torch.arange(8) * 3, torch.arange(8)] = 1000.0
    loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
    with MlpLoss(rows, 8, 200, "bf16", grad=False) as layer:
        layer.forward(x, w, at * 3, loss, lse)
        torch.cuda.synchronize()
    want = math.log1p(199 * math.exp(-8.0))
    assert float((loss.double() - want).abs().max()) <= 2e-6
    assert float((lse.double() - 1000 - want).abs().max()) <= 2.0 ** -14


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


# ------------------------------------------------- forced plans, pieces, far apart

@pytest.mark.parametrize("rows,H,V", [(9, 64, 100), (300, 72, 777)])
def test_loss_backward_of_the_lse_alone_and_ones(rows, H, V):
    check_loss_backward(rows, H, V, "bf16", dloss=None, dlse=True)
    check_loss_backward(rows, H, V, "f16", dloss=None, dlse=True)


@pytest.mark.parametrize("left_out", ["some", "none", "all"])
@pytest.mark.parametrize("rows", [4095, 4096, 4097, 9001])
def test_loss_of_many_rows(rows, left_out):
    """Rows are packed a thousand at a time."""
    check_loss_forward(rows, 16, 100, "bf16", left_out)
    check_loss_backward(rows, 16, 100, "bf16", left_out, dloss="any", dlse=True)


@pytest.mark.parametrize("plan", [0, 1, 2, 3, 4, 5, 6])
@pytest.mark.parametrize("rows,H,V", [(33, 136, 300), (300, 200, 700), (777, 72, 513)])
def test_loss_forward_with_every_tile(rows, H, V, plan):
    check_loss_forward(rows, H, V, "bf16", plan=plan)


@pytest.mark.parametrize("split", [1, 3, 8])
@pytest.mark.parametrize("plan", [1, 2, 3, 4, 5, 6])
def test_loss_backward_with_every_tile(plan, split):
    for rows, H, V in ((33, 136, 1300), (300, 200, 2100), (777, 72, 513)):
        check_loss_backward(rows, H, V, "f16", plan=plan, split=split)


@pytest.mark.parametrize("rows", [257, 320, 321, 352, 448, 480, 481, 512, 670, 700])
def test_loss_with_tall_tiles(rows):
    """Row counts around what tiles of 160 to 256 rows take, all rows counted and some."""
    for left_out in ("none", "some"):
        check_loss_forward(rows, 136, 1500, "bf16", left_out, plan=4)
        check_loss_backward(rows, 136, 1500, "bf16", left_out, plan=4)


@pytest.mark.parametrize("rows,H", [(1, 2048), (40, 4096), (200, 2104), (257, 4096)])
def test_loss_of_long_rows(rows, H):
    """Reductions that begin at another place for each tile."""
    for dtype in ("f16", "bf16"):
        check_loss_forward(rows, H, 1000, dtype)
        check_loss_backward(rows, H, 1000, dtype)


def test_loss_backward_in_pieces():
    """A vocabulary whose dz does not fit the workspace at once, the last piece ragged."""
    check_loss_backward(3000, 64, 50001, "bf16")


def test_loss_backward_in_many_pieces():
    """A handle for far more rows than the call has, and one whose pieces are 256 words wide."""
    check_loss_backward(700, 64, 50001, "f16", most=1 << 16)
    check_loss_backward(600, 64, 1001, "f16", most=1 << 20)


def test_loss_of_a_head_past_2_gb():
    """Offsets of W and dW past 2^31 bytes."""
    rows, H, V = 20, 8192, 140000
    g, n = gen(5)
    x = n(rows, H).bfloat16()
    w = torch.empty(V, H, dtype=torch.bfloat16, device="cuda")
    for v in range(0, V, 20000):
        w[v:v + 20000].copy_(n(20000, H) * (3 / math.sqrt(H)))
    target = torch.randint(V - 1000, V, (rows,), generator=g, device="cuda")
    loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    with MlpLoss(rows, H, V, "bf16") as layer:
        layer.forward(x, w, target, loss, lse)
        layer.backward(x, w, target, lse, dx=dx, dw=dw)
        torch.cuda.synchronize()
    z = torch.cat([x.double() @ w[v:v + 20000].double().t().contiguous() for v in range(0, V, 20000)], 1)
    ez = (H / 32 + 64) * E32 * H * float(x.abs().amax()) * float(w.abs().amax()) / 4
    ref = torch.logsumexp(z, 1)
    close(lse, ref, ez + 2.0 ** -18 + 2 * E32 * ref.abs(), "lse")
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(rows, device="cuda"), target] -= 1.0
    for v in range(0, V, 20000):
        part = dz[:, v:v + 20000]
        want = part.t().contiguous() @ x.double()
        size = part.abs().t().contiguous() @ x.double().abs()
        close(dw[v:v + 20000], want, U["bf16"] * want.abs() + (U["bf16"] + 2.0 ** -16) * size, "dw")


# ------------------------------------------------------------- values and rows

def run_loss(x, w, target, dtype, dloss=None, dlse=None, layer=None):
    rows, V = x.shape[0], w.shape[0]
    loss, lse = (torch.full((rows,), 7.0, device="cuda") for _ in range(2))
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    own = layer is None
    layer = layer or MlpLoss(rows, x.shape[1], V, dtype)
    layer.forward(x, w, target, loss, lse)
    layer.backward(x, w, target, lse, dloss, dlse, dx=dx, dw=dw)
    torch.cuda.synchronize()
    if own:
        layer.close()
    return loss, lse, dx, dw


@pytest.mark.parametrize("rows", [5, 300, 700])
def test_rows_left_out_may_hold_anything(rows):
    """NaN and infinities in rows that are left out, and a NaN in their dloss, reach nothing."""
    x, w, target = loss_case(rows, 72, 500, "bf16", 3)
    target[1] = -5
    out = target < 0
    clean = x.clone()
    clean[out] = 0
    d = torch.rand(rows, device="cuda")
    x[out] = math.nan
    x[out.nonzero()[0]] = math.inf
    got = run_loss(x, w, target, "bf16", torch.where(out, math.nan, d))
    want = run_loss(clean, w, target, "bf16", torch.where(out, 0.0, d))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [5, 300])
def test_a_row_that_is_not_finite(rows):
    """It has a loss and a dx that are not finite, and so has dW; the other rows' are what they would be."""
    x, w, target = loss_case(rows, 72, 500, "bf16", 4, "none")
    want = run_loss(x, w, target, "bf16")
    x[2, 5] = math.nan
    loss, lse, dx, dw = run_loss(x, w, target, "bf16")
    others = torch.arange(rows, device="cuda") != 2
    assert loss[2].isnan() and lse[2].isnan() and dx[2].isnan().all() and dw.isnan().any()
    assert torch.equal(loss[others], want[0][others]) and torch.equal(lse[others], want[1][others])
    assert torch.equal(dx[others], want[2][others])


@pytest.mark.parametrize("rows", [5, 300])
def test_targets_outside_the_vocabulary(rows):
    """Shown as NaN; in the gradient their rows are left out."""
    x, w, target = loss_case(rows, 72, 500, "f16", 5, "none")
    wrong = target.clone()
    wrong[1], wrong[3], wrong[4] = 500, 2 ** 40, 2 ** 31
    left = torch.where(wrong >= 500, -1, wrong)
    got, want = run_loss(x, w, wrong, "f16"), run_loss(x, w, left, "f16")
    outside = wrong >= 500
    for k in range(2):
        assert got[k][outside].isnan().all() and torch.equal(got[k][~outside], want[k][~outside])
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
    low = torch.where(wrong >= 500, -2 ** 62, wrong)
    for a, b in zip(run_loss(x, w, low, "f16"), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [6, 300])
def test_upstream_gradients_of_zero_and_almost_zero(rows, dtype):
    x, w, target = loss_case(rows, 72, 500, dtype, 6, "none")
    for value in (0.0, 1e-42, 1e-38, 2.0 ** -126):
        _, _, dx, dw = run_loss(x, w, target, dtype, torch.full((rows,), value, device="cuda"))
        assert dx.isfinite().all() and dw.isfinite().all()
        assert float(dx.abs().max()) <= 2.0 ** -100


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dtype,value", [("f16", 1e5), ("f16", 2.0 ** -10), ("bf16", 1e5)])
@pytest.mark.parametrize("rows", [6, 300])
def test_an_upstream_gradient_that_is_not_finite(rows, dtype, value, bad):
    """Its row's dx is not finite, nor is dW; the other rows' dx is what it would be: dz's unit is theirs."""
    x, w, target = loss_case(rows, 72, 500, dtype, 8, "none", spread=0.1)
    d = torch.full((rows,), value, device="cuda")
    d[2] = 0.0
    want = run_loss(x, w, target, dtype, d)[2]
    others = torch.arange(rows, device="cuda") != 2
    assert want.isfinite().all() and want[others].any(1).all()
    zeros = torch.zeros_like(d)
    for dloss, dlse in ((torch.where(others, d, bad), None), (d, torch.where(others, zeros, bad))):
        _, _, dx, dw = run_loss(x, w, target, dtype, dloss, dlse)
        assert not dx[2].isfinite().any() and not dw.isfinite().any()
        assert torch.equal(dx[others], want[others])


@pytest.mark.parametrize("rows", [6, 300])
def test_upstream_gradients_of_very_different_sizes(rows):
    """bf16 holds each row's dz whatever the others' size."""
    d = torch.logspace(-30, 0, rows, device="cuda")
    x, w, target = loss_case(rows, 72, 500, "bf16", 7, "none")
    _, lse, dx, _ = run_loss(x, w, target, "bf16", d)
    z, _, _, _ = loss_ref(x, w, target)
    dz = torch.exp(z - lse.double()[:, None])
    dz[torch.arange(rows, device="cuda"), target] -= 1.0
    ref = (dz @ w.double()) * d.double()[:, None]
    size = (dz.abs() @ w.double().abs()) * d.double()[:, None]
    close(dx, ref, U["bf16"] * ref.abs() + (U["bf16"] + 2.0 ** -14) * size, "dx")


@pytest.mark.parametrize("which", ["dx", "dw"])
@pytest.mark.parametrize("rows,H,V", [(7, 40, 33), (300, 64, 129)])
def test_loss_gradient_against_differences(rows, H, V, which):
    """The directional derivative of sum(a loss + b lse) by central differences in 64 bits."""
    x, w, target = loss_case(rows, H, V, "f16", 8)
    _, n = gen(1)
    a, b = n(rows), n(rows)
    _, _, dx, dw = run_loss(x, w, target, "f16", a, b)
    got = {"dx": dx, "dw": dw}[which].double()
    d = torch.randn(got.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.float64)

    def value(t):
        _, lse, loss, _ = loss_ref(x.double() + (t * d if which == "dx" else 0), w.double() + (t * d if which == "dw" else 0), target)
        return (a.double() * loss + b.double() * lse).sum()
    h = 1e-5
    diff = float((value(h) - value(-h)) / (2 * h))
    # roundings of outputs and of dz, each of at most u |g d|, independent: eight times their 2-norm
    assert abs(float((got * d).sum()) - diff) <= 8 * 2 * U["f16"] * float((got * d).norm()) + 1e-4


def test_loss_of_no_rows():
    w = torch.randn(300, 64, device="cuda").half()
    dw = torch.full_like(w, 7.0)
    with MlpLoss(8, 64, 300, "f16") as layer:
        e = torch.empty(0, 64, dtype=torch.float16, device="cuda")
        f, t = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
        layer.forward(e, w, t, f, f)
        layer.backward(e, w, t, f, dx=e, dw=dw)
        torch.cuda.synchronize()
    assert (dw == 0).all()


# --------------------------------------------------- streams, graphs, repetition

@pytest.mark.parametrize("rows", [20, 300, 700])
def test_loss_twice_the_same_and_with_fewer_rows(rows):
    """A handle's calls depend on nothing from earlier ones: other rows, other targets, then the first again."""
    x, w, target = loss_case(rows, 136, 1003, "bf16", 9)
    with MlpLoss(rows, 136, 1003, "bf16") as layer:
        first = run_loss(x, w, target, "bf16", layer=layer)
        run_loss(x[:rows // 2], w, torch.zeros_like(target[:rows // 2]), "bf16", layer=layer)
        run_loss(x[:3], w, torch.full_like(target[:3], -1), "bf16", layer=layer)
        again = run_loss(x, w, target, "bf16", layer=layer)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_loss_on_two_streams_at_once():
    """Separate handles on streams of their own."""
    cases = [loss_case(r, 136, 1003, "bf16", 10 + r) for r in (40, 500)]
    want = [run_loss(*c, "bf16") for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    layers = [MlpLoss(c[0].shape[0], 136, 1003, "bf16") for c in cases]
    outs = [[torch.empty(c[0].shape[0], device="cuda") for _ in range(2)] + [torch.empty_like(c[0]), torch.empty_like(c[1])] for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for (x, w, t), s, layer, (loss, lse, dx, dw) in zip(cases, streams, layers, outs):
            with torch.cuda.stream(s):
                layer.forward(x, w, t, loss, lse)
                layer.backward(x, w, t, lse, dx=dx, dw=dw)
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    for layer in layers:
        layer.close()


@pytest.mark.parametrize("rows", [20, 700])
def test_loss_graph_replays(rows):
    """Captured once, replayed with other inputs and targets, eager work between the replays."""
    x, w, target = loss_case(rows, 136, 1003, "bf16", 12)
    loss, lse = (torch.empty(rows, device="cuda") for _ in range(2))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    with MlpLoss(rows, 136, 1003, "bf16") as layer:
        def step():
            layer.forward(x, w, target, loss, lse)
            layer.backward(x, w, target, lse, dx=dx, dw=dw)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for k in range(3):
            x2, w2, t2 = loss_case(rows, 136, 1003, "bf16", 20 + k, ("some", "none", "all")[k])
            x.copy_(x2), w.copy_(w2), target.copy_(t2)
            for t in (loss, lse, dx, dw):
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((loss, lse, dx, dw), run_loss(x2, w2, t2, "bf16")):
                assert torch.equal(a, b)


def test_loss_refusals_of_tensors():
    x, w, target = loss_case(6, 64, 100, "f16", 1)
    loss, lse = (torch.empty(6, device="cuda") for _ in range(2))
    with MlpLoss(6, 64, 100, "f16", grad=False) as layer:
        with pytest.raises(ValueError, match="shape"):
            layer.forward(x[:, :56], w, target, loss, lse)
        with pytest.raises(ValueError, match="w has shape"):
            layer.forward(x, w[:50], target, loss, lse)
        with pytest.raises(ValueError, match="w has shape"):
            layer.forward(x, w.t(), target, loss, lse)
        with pytest.raises(ValueError, match="f16"):
            layer.forward(x.bfloat16(), w, target, loss, lse)
        with pytest.raises(ValueError, match="int64"):
            layer.forward(x, w, target.int(), loss, lse)
        with pytest.raises(ValueError, match="float32"):
            layer.forward(x, w, target, loss.half(), lse)
        with pytest.raises(ValueError, match="target must be"):
            layer.forward(x, w, target[:5], loss, lse)
        with pytest.raises(ValueError, match="device"):
            layer.forward(x, w, target.cpu(), loss, lse)
        with pytest.raises(MlpChainError, match="lse"):
            layer.forward(x, w, target, loss, None)
        with pytest.raises(MlpChainError, match="gradient"):
            layer.backward(x, w, target, lse, dx=torch.empty_like(x))
        with pytest.raises(MlpChainError, match="aligned"):
            off = torch.empty(6 * 64 + 8, dtype=torch.float16, device="cuda")[4:6 * 64 + 4].view(6, 64)
            layer.forward(off, w, target, loss, lse)
        with pytest.raises(MlpChainError, match="rows"):
            big = torch.cat([x, x])
            layer.forward(big, w, torch.cat([target, target]), torch.cat([loss, loss]), torch.cat([lse, lse]))
