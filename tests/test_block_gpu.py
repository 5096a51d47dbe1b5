"""Layer norm, linear layer and the whole pre-norm block on the GPU, through
the binding, against the definitions in 64 bits.

Tolerances.  u is the storage type's unit roundoff (11 and 8 significant bits:
2^-11 fp16, 2^-8 bf16) and every output is rounded once: u |ref|, plus fp16's half subnormal step.
An fp32 sum of n terms in chains of at most n/32 + 64 additions errs by at
most (n/32 + 64) 2^-23 sum|terms| (matrix cores truncate, so 2^-23 each).
Elementwise fp32 arithmetic (a handful of operations, hardware 2^x and
reciprocal) errs by 2^-20 of its largest term.  dz is rounded to the storage
type before the gradient's products; the reference rounds its own dz the
same way, and where the two fp32 values fall on either side of a rounding
boundary (a chance of about 2^-20 / u per element) they differ by 2u: a few
such elements in one sum are allowed for.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import mlp_block as mb  # noqa: E402
from consumer_gemm_chain_amd import MlpBlock, MlpChainError, MlpLinear, MlpNorm  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
E32 = 2.0 ** -23
EPS = 1e-5


def gen(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g, device="cuda")


def padded(t, pad):
    """`t` as a view with `pad` more elements per row, which hold NaN."""
    if t is None or pad == 0:
        return t
    base = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = base[:, : t.shape[1]]
    view.copy_(t)
    return view


def empty(rows, cols, dtype, pad=0):
    """An output filled with a canary, and a check that its padding still holds it."""
    base = torch.full((rows, cols + pad), 77.0, dtype=DT[dtype], device="cuda")
    return base[:, :cols], lambda: bool((base[:, cols:] == 77.0).all())


def close(got, ref, tol, what):
    got = got.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(got[bad][0]), float(ref[bad][0]),
                           float(torch.as_tensor(tol).expand_as(ref)[bad][0]))


def rounded(ref, dtype):
    return U[dtype] * ref.abs() + TINY[dtype]


# ------------------------------------------------------------------------ norm

def norm_case(rows, H, dtype, seed, offset=0.0):
    n = gen(seed)
    dt = DT[dtype]
    return ((offset + n(rows, H) * (0.5 + n(H).abs())).to(dt), (1 + 0.1 * n(H)).to(dt), (0.1 * n(H)).to(dt),
            (0.1 * n(rows, H)).to(dt), (0.1 * n(rows, H)).to(dt))


def norm_ref(x, w, b):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
    xhat = c * rstd[:, None]
    y = xhat * (w.double() if w is not None else 1) + (b.double() if b is not None else 0)
    return y, mean, rstd, xhat


def check_norm_forward(rows, H, dtype, pad=0, offset=0.0, affine="wb", seed=1):
    x, w, b, _, _ = norm_case(rows, H, dtype, seed, offset)
    w, b = (w if "w" in affine else None), (b if "b" in affine else None)
    y, ok = empty(rows, H, dtype, pad)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    with MlpNorm(H, dtype, EPS) as layer:
        layer.forward(padded(x, pad), w, b, y, mean, rstd)
        torch.cuda.synchronize()
    ry, rm, rr, xhat = norm_ref(x, w, b)
    big = x.double().abs().amax(1) * rr                       # cancellation in x - mean
    chain = (H / 32 + 64) * E32
    close(mean, rm, chain * x.double().abs().mean(1), "mean")
    close(rstd, rr, rr * (chain + 4 * (chain * big) ** 2 + 2.0 ** -20), "rstd")
    wabs = w.double().abs() if w is not None else 1.0
    tol32 = wabs * (xhat.abs() * (chain + 4 * (chain * big[:, None]) ** 2) + chain * big[:, None]) + 2.0 ** -20 * (ry.abs() + xhat.abs() * wabs)
    close(y, ry, rounded(ry, dtype) + tol32, "y")
    assert ok(), "padding was written"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H", [(1, 1), (3, 2), (2, 7), (5, 8), (1, 512), (9, 65), (130, 512), (3, 1000), (2, 2056),
                                    (67, 4096), (5, 8192), (3, 12288), (2, 16384), (2, 16392), (2, 40001), (1500, 264)])
def test_norm_forward(rows, H, dtype):
    check_norm_forward(rows, H, dtype)


@pytest.mark.parametrize("rows,H,pad", [(5, 512, 8), (5, 512, 3), (7, 1003, 5), (3, 12288, 64), (4, 8192, 1)])
def test_norm_forward_strides(rows, H, pad):
    check_norm_forward(rows, H, "f16", pad)
    check_norm_forward(rows, H, "bf16", pad)


@pytest.mark.parametrize("affine", ["", "w", "b"])
@pytest.mark.parametrize("H", [77, 1024])
def test_norm_forward_without_scale_or_shift(affine, H):
    check_norm_forward(6, H, "f16", affine=affine)


@pytest.mark.parametrize("H", [100, 8192])
def test_norm_forward_far_from_zero(H):
    """A mean a thousand standard deviations from zero: the variance comes from centred values."""
    check_norm_forward(4, H, "f16", offset=1000.0)


@pytest.mark.parametrize("H", [24, 333, 8192])
def test_norm_of_constant_and_broken_rows(H):
    """A constant row gives the shift; a row with NaN or infinity gives NaN and leaves the others alone."""
    x, w, b, _, _ = norm_case(5, H, "f16", 3)
    x[1] = 3.0
    x[2, H // 2] = float("nan")
    x[3, 0] = float("inf")
    y = torch.empty_like(x)
    with MlpNorm(H, "f16", EPS) as layer:
        layer.forward(x, w, b, y)
    assert torch.equal(y[1], b)
    assert y[2].isnan().all() and y[3].isnan().all()
    ry, _, _, _ = norm_ref(x[[0, 4]], w, b)
    close(y[[0, 4]], ry, rounded(ry, "f16") + 2.0 ** -12, "other rows")


def norm_grad_ref(dy, x, w, mean, rstd, dres):
    dy, x = dy.double(), x.double()
    xhat = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy * w.double() if w is not None else dy
    m0, m1 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd.double()[:, None] * (g - m0 - xhat * m1)
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xhat).sum(0), dy.sum(0), xhat, g, m0, m1


def check_norm_backward(rows, H, dtype, pad=0, dres=True, weight=True, seed=2, offset=0.0, in_place=False):
    x, w, b, dy, dr = norm_case(rows, H, dtype, seed, offset)
    w, dr = (w if weight else None), (dr if dres else None)
    _, mean, rstd, _ = norm_ref(x, w, b)
    mean, rstd = mean.float(), rstd.float()
    dx, ok = empty(rows, H, dtype, pad)
    dres_in = padded(dr, pad)
    if in_place:
        dx.copy_(dr)
        dres_in = dx
    dw, db = (torch.full((H,), 77.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    with MlpNorm(H, dtype, EPS) as layer:
        layer.backward(padded(dy, pad), padded(x, pad), w, mean, rstd, dx, dw, db, dres=dres_in)
        torch.cuda.synchronize()
    rdx, rdw, rdb, xhat, g, m0, m1 = norm_grad_ref(dy, x, w, mean, rstd, dr)
    chain = (H / 32 + 64) * E32
    r = rstd.double()[:, None]
    big = 1 + x.double().abs().amax(1, keepdim=True) * r     # cancellation in x - mean
    sums = g.abs().mean(1, keepdim=True) * chain + (g * xhat).abs().mean(1, keepdim=True) * chain * xhat.abs()
    tol32 = r * (sums + 2.0 ** -20 * (g.abs() + m0.abs() + big * (m1.abs() * (1 + xhat.abs()) + g.abs().mean(1, keepdim=True) * xhat.abs())))
    close(dx, rdx, rounded(rdx, dtype) + tol32 + 2.0 ** -22 * rdx.abs(), "dx")
    cols = (rows / 32 + 64) * E32
    close(dw, rdw, rounded(rdw, dtype) + (dy.double().abs() * (cols * xhat.abs() + 2.0 ** -21 * big)).sum(0), "dweight")
    close(db, rdb, rounded(rdb, dtype) + cols * dy.double().abs().sum(0), "dbias")
    assert ok(), "padding was written"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H", [(1, 1), (3, 2), (2, 7), (5, 8), (1, 512), (9, 65), (64, 512), (257, 1000), (2, 2056),
                                    (700, 4096), (300, 8192), (33, 12288), (2, 16384), (3, 16392), (2, 40001), (1500, 264)])
def test_norm_backward(rows, H, dtype):
    check_norm_backward(rows, H, dtype)


@pytest.mark.parametrize("rows,H,pad", [(5, 512, 8), (5, 512, 3), (70, 1003, 5), (3, 12288, 64), (4, 8192, 1)])
@pytest.mark.parametrize("dres", [False, True])
def test_norm_backward_strides(rows, H, pad, dres):
    check_norm_backward(rows, H, "f16", pad, dres)
    check_norm_backward(rows, H, "bf16", pad, dres)


@pytest.mark.parametrize("H", [77, 1024])
def test_norm_backward_variants(H):
    check_norm_backward(40, H, "f16", weight=False)
    check_norm_backward(40, H, "bf16", in_place=True)
    check_norm_backward(4, H, "f16", offset=100.0)


@pytest.mark.parametrize("rows,H", [(48, 512), (49, 512), (2, 512), (12, 2041), (13, 2041), (3, 8192), (4, 8192)])
def test_norm_backward_of_a_single_workgroup(rows, H):
    """The row counts around the last one that a single workgroup takes; its outputs one at a time."""
    check_norm_backward(rows, H, "bf16")
    x, w, b, dy, _ = norm_case(rows, H, "f16", 4)
    _, mean, rstd, _ = norm_ref(x, w, b)
    out = [[torch.full((n, H) if n else (H,), 7.0, dtype=x.dtype, device="cuda") for n in (rows, 0, 0)] for _ in range(4)]
    with MlpNorm(H, "f16", EPS) as layer:
        for (dx, dw, db), keep in zip(out, ((1, 1), (1, 0), (0, 1), (0, 0))):
            layer.backward(dy, x, w, mean.float(), rstd.float(), dx, dw if keep[0] else None, db if keep[1] else None)
        torch.cuda.synchronize()
    for (dx, dw, db), keep in zip(out, ((1, 1), (1, 0), (0, 1), (0, 0))):
        assert torch.equal(dx, out[0][0])
        assert torch.equal(dw, out[0][1]) if keep[0] else (dw == 7).all()
        assert torch.equal(db, out[0][2]) if keep[1] else (db == 7).all()


@pytest.mark.parametrize("H", [40, 333])
@pytest.mark.parametrize("which", ["dx", "dweight", "dbias"])
def test_norm_gradient_against_differences(H, which):
    """The directional derivative of sum(dy norm(x)) by central differences in 64 bits."""
    rows = 6
    x, w, b, dy, _ = norm_case(rows, H, "f16", 8)
    _, mean, rstd, _ = norm_ref(x, w, b)
    dx = torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    with MlpNorm(H, "f16", EPS) as layer:
        layer.backward(dy, x, w, mean.float(), rstd.float(), dx, dw, db)
    at = {"dx": x, "dweight": w, "dbias": b}
    got = {"dx": dx, "dweight": dw, "dbias": db}[which].double()
    d = torch.randn(got.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.float64)

    def loss(t):
        v = {k: p.double() + (t * d if k == which else 0) for k, p in at.items()}
        return (dy.double() * norm_ref(v["dx"], v["dweight"], v["dbias"])[0]).sum()
    h = 1e-5
    diff = float((loss(h) - loss(-h)) / (2 * h))
    # independent roundings of at most u |g d| each: eight times their 2-norm, and the difference's own error
    assert abs(float((got * d).sum()) - diff) <= 8 * U["f16"] * float((got * d).norm()) + 1e-6


def test_norm_outputs_left_out():
    x, w, b, dy, dr = norm_case(10, 512, "f16", 4)
    y, y2, dx, dx2 = (torch.empty_like(x) for _ in range(4))
    mean, rstd = torch.empty(10, device="cuda"), torch.empty(10, device="cuda")
    dw, db, dw2, db2 = (torch.empty_like(w) for _ in range(4))
    with MlpNorm(512, "f16", EPS) as layer:
        layer.forward(x, w, b, y, mean, rstd)
        layer.forward(x, w, b, y2)
        layer.backward(dy, x, w, mean, rstd, dx, dw, db)
        layer.backward(dy, x, w, mean, rstd, dx2)
        layer.backward(dy, x, w, mean, rstd, dx2, dweight=dw2)
        layer.backward(dy, x, w, mean, rstd, dx2, dbias=db2)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_norm_offsets_past_32_bits():
    """Rows 2^24 elements apart: byte offsets past 2^32."""
    H, rows, ld = 264, 140, 1 << 24
    x, w, b, dy, _ = norm_case(rows, H, "f16", 5)
    far = torch.empty(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)[:, :H]
    far.copy_(x)
    y, y2, dx, dx2 = (torch.empty_like(x) for _ in range(4))
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    with MlpNorm(H, "f16", EPS) as layer:
        layer.forward(x, w, b, y, mean, rstd)
        layer.forward(far, w, b, y2)
        layer.backward(dy, x, w, mean, rstd, dx)
        layer.backward(dy, far, w, mean, rstd, dx2)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
        layer.forward(x, w, b, far)
        assert torch.equal(y, far)


# ---------------------------------------------------------------------- linear

def gelu(h):
    return 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h ** 3)))


def act_ref(h, act, N):
    if act == "gelu_tanh":
        return gelu(h)
    if act == "swiglu":
        return h[:, :N] * torch.sigmoid(h[:, :N]) * h[:, N:]
    return h


def linear_case(rows, K, N, act, dtype, seed):
    n, dt = gen(seed), DT[dtype]
    gN = N * (2 if act == "swiglu" else 1)
    return {"x": n(rows, K).to(dt), "w": (n(K, gN) / math.sqrt(K)).to(dt), "bias": (0.3 * n(gN)).to(dt),
            "res": n(rows, N).to(dt), "dy": (0.1 * n(rows, N)).to(dt), "z": n(rows, gN).to(dt), "gN": gN}


def check_linear_forward(rows, K, N, act="none", dtype="f16", bias=True, res=True, save=True, pad=0, in_place=False,
                         seed=11):
    c = linear_case(rows, K, N, act, dtype, seed)
    gN = c["gN"]
    y, ok = empty(rows, N, dtype, pad)
    z, okz = empty(rows, gN, dtype, pad)
    r = padded(c["res"], pad) if res else None
    if in_place:
        y.copy_(c["res"])
        r = y
    with MlpLinear(rows, K, N, act, dtype) as layer:
        layer.forward(padded(c["x"], pad), padded(c["w"], pad), y, bias=c["bias"] if bias else None, residual=r,
                      z=z if save else None)
        torch.cuda.synchronize()
    x, w = c["x"].double(), c["w"].double()
    h = torch.mm(x, w) + (c["bias"].double() if bias else 0)
    th = (K / 32 + 64) * E32 * (torch.mm(x.abs(), w.abs()) + c["bias"].double().abs()) + 2.0 ** -22 * h.abs()
    a = act_ref(h, act, N)
    if act == "swiglu":
        g, u = h[:, :N], h[:, N:]
        ta = 1.1 * th[:, :N] * u.abs() + (g * torch.sigmoid(g)).abs() * th[:, N:] + 1.1 * th[:, :N] * th[:, N:]
    else:
        ta = 1.2 * th
    ref = a + (c["res"].double() if res else 0)
    close(y, ref, rounded(ref, dtype) + ta + 2.0 ** -20 * (a.abs() + ref.abs()), "y")
    assert ok(), "padding was written"
    if save:
        close(z, h, rounded(h, dtype) + th, "z")
        assert okz(), "padding of z was written"


SIZES = [(1, 8, 8), (1, 512, 2048), (3, 72, 40), (15, 256, 136), (16, 520, 264), (17, 64, 128), (31, 1032, 72),
         (64, 512, 512), (65, 2056, 200), (128, 128, 1480), (129, 776, 264), (255, 320, 512), (257, 264, 776),
         (300, 1000, 600), (513, 512, 520), (1000, 136, 1032)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows,K,N", SIZES)
def test_linear_forward(rows, K, N, act, dtype):
    check_linear_forward(rows, K, N, act, dtype)


@pytest.mark.parametrize("bias,res,save", [(b, r, s) for b in (0, 1) for r in (0, 1) for s in (0, 1)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
def test_linear_forward_options(bias, res, save, act):
    check_linear_forward(40, 264, 328, act, "f16", bool(bias), bool(res), bool(save), pad=8)
    check_linear_forward(300, 264, 328, act, "bf16", bool(bias), bool(res), bool(save), pad=64)


@pytest.mark.parametrize("rows", [5, 200])
def test_linear_forward_in_place(rows):
    check_linear_forward(rows, 512, 264, "none", "f16", in_place=True)


@pytest.mark.parametrize("rows,K,N,act,dtype", [(1, 12288, 6144, "gelu_tanh", "f16"), (16, 3584, 8192, "none", "bf16"),
                                                (4, 8192, 2752, "swiglu", "f16"), (64, 12288, 6144, "gelu_tanh", "bf16"),
                                                (300, 8192, 2752, "swiglu", "f16"), (515, 6144, 12288, "none", "f16"),
                                                (2048, 6144, 12288, "none", "f16")])
def test_linear_forward_model_sizes(rows, K, N, act, dtype):
    check_linear_forward(rows, K, N, act, dtype)


def dz_ref(dy, z, act, N):
    dy = dy.double()
    if act == "none":
        return dy
    z = z.double().requires_grad_()
    g, = torch.autograd.grad(act_ref(z, act, N), z, dy)
    return g


def check_linear_backward(rows, K, N, act="none", dtype="f16", pad=0, seed=21):
    c = linear_case(rows, K, N, act, dtype, seed)
    gN = c["gN"]
    dx, okx = empty(rows, K, dtype, pad)
    dw, okw = empty(K, gN, dtype, pad)
    db = torch.full((gN,), 77.0, dtype=DT[dtype], device="cuda")
    z = padded(c["z"], pad) if act != "none" else None
    with MlpLinear(rows, K, N, act, dtype) as layer:
        layer.backward(padded(c["dy"], pad), padded(c["x"], pad), padded(c["w"], pad), dx=dx, dw=dw, db=db, z=z)
        torch.cuda.synchronize()
    x, w = c["x"].double(), c["w"].double()
    dz = dz_ref(c["dy"], c["z"], act, N)
    dzr = dz.to(DT[dtype]).double()
    flip = 0.0 if act == "none" else 4 * 2 * U[dtype] * float(dzr.abs().max())
    ref = torch.mm(dzr, w.t())
    tol = (gN / 32 + 64) * E32 * torch.mm(dzr.abs(), w.abs().t()) + flip * float(w.abs().max())
    close(dx, ref, rounded(ref, dtype) + tol, "dx")
    ref = torch.mm(x.t(), dzr)
    tol = (rows / 32 + 64) * E32 * torch.mm(x.abs().t(), dzr.abs()) + flip * float(x.abs().max())
    close(dw, ref, rounded(ref, dtype) + tol, "dw")
    ref = dz.sum(0)
    # db sums dz before its rounding; the largest term of dz is |dy| (1 + |z|)^2
    largest = c["dy"].double().abs() * (1 + c["z"].double()[:, :N].abs()) * (1 + c["z"].double()[:, -N:].abs())
    largest = largest.repeat(1, gN // N)
    close(db, ref, rounded(ref, dtype) + (rows / 32 + 64) * E32 * dz.abs().sum(0) + 2.0 ** -20 * largest.sum(0), "db")
    assert okx() and okw(), "padding was written"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows,K,N", SIZES)
def test_linear_backward(rows, K, N, act, dtype):
    check_linear_backward(rows, K, N, act, dtype)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows,pad", [(40, 8), (300, 64), (63, 16)])
def test_linear_backward_strides(rows, pad, act):
    check_linear_backward(rows, 264, 328, act, "f16", pad)


@pytest.mark.parametrize("rows,K,N,act,dtype", [(1, 12288, 6144, "gelu_tanh", "f16"), (300, 8192, 2752, "swiglu", "f16"),
                                                (1000, 8192, 3584, "swiglu", "bf16"), (515, 6144, 12288, "none", "f16"),
                                                (2048, 12288, 6144, "gelu_tanh", "f16")])
def test_linear_backward_model_sizes(rows, K, N, act, dtype):
    check_linear_backward(rows, K, N, act, dtype)


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
def test_linear_gradient_against_differences(act):
    """Directional derivatives of sum(dy act(x W + b)) in x, W and b by central differences in 64 bits."""
    rows, K, N = 20, 72, 40
    c = linear_case(rows, K, N, act, "f16", 31)
    x, w, b = (c[k].double() for k in ("x", "w", "bias"))
    z = (torch.mm(x, w) + b).half()
    dx, dw, db = torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["bias"])
    with MlpLinear(rows, K, N, act, "f16") as layer:
        layer.backward(c["dy"], c["x"], c["w"], dx=dx, dw=dw, db=db, z=z)
    dy = c["dy"].double()
    # the kernels differentiate at the rounded z: the differences are taken around the same point
    shift = z.double() - (torch.mm(x, w) + b)
    for k, got in (("x", dx), ("w", dw), ("b", db)):
        d = torch.randn(got.shape, generator=torch.Generator("cuda").manual_seed(2), device="cuda", dtype=torch.float64)

        def loss(t):
            v = {"x": x, "w": w, "b": b}
            v[k] = v[k] + t * d
            return (dy * act_ref(torch.mm(v["x"], v["w"]) + v["b"] + shift, act, N)).sum()
        h = 1e-5
        diff = float((loss(h) - loss(-h)) / (2 * h))
        got = got.double()
        assert abs(float((got * d).sum()) - diff) <= 8 * 2 * U["f16"] * float((got * d).norm()) + 1e-6, k


@pytest.mark.parametrize("act", ["gelu_tanh", "swiglu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_activation_gradient_at_extremes(act, dtype):
    """dz, read off db for a single row, at z from the type's largest values to zero: finite and right; NaN stays NaN."""
    big = 6e4 if dtype == "f16" else 3e38
    v = torch.tensor([0.0, -0.0, 1e-7, -1e-7, 1, -1, 5, -5, 11.9, -11.9, 12.1, -12.1, 100, -100, big, -big],
                     device="cuda", dtype=torch.float64).to(DT[dtype])
    N = 16
    z = v[None] if act == "gelu_tanh" else torch.cat([v[None], torch.ones_like(v)[None]], 1)
    dy = torch.ones((1, N), dtype=DT[dtype], device="cuda")
    db = torch.empty(z.shape[1], dtype=DT[dtype], device="cuda")
    with MlpLinear(1, 8, N, act, dtype) as layer:
        layer.backward(dy, None, None, db=db, z=z.contiguous())
        s = torch.sigmoid(v.double())
        if act == "gelu_tanh":
            t = v.double().clamp(-40, 40)
            sg = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
            ref = sg + t * sg * (1 - sg) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * t * t)
        else:
            ref = torch.cat([torch.where(v.abs() > 1e4, (v > 0).double(), s + v.double() * s * (1 - s)), v.double() * s])
        close(db, ref, rounded(ref, dtype) + 2.0 ** -18, "dz")
        z2 = z.clone()
        z2[0, 3] = float("nan")
        layer.backward(dy, None, None, db=db, z=z2)
        assert db[3].isnan() and not db[4:N].isnan().any()


CONFIGS = range(8)


@pytest.mark.parametrize("dtype,rows,K,N", [("f16", 150, 328, 264), ("bf16", 300, 640, 136), ("f16", 9, 200, 72)])
def test_every_tile_configuration_gives_the_same_bits(dtype, rows, K, N):
    """Unsplit, every configuration adds the same products in the same order; split in equal parts likewise."""
    c = linear_case(rows, K, N, "swiglu", dtype, 9)
    x, w, b, dy, z = c["x"], c["w"], c["bias"], c["dy"], c["z"]
    # (a handle of 150 rows at least: its workspace holds the forced plans' partials)
    with MlpLinear(max(rows, 150), K, N, "swiglu", dtype) as layer:
        results = {}
        for split in (1, 2, 4):
            seen = results[split] = [None] * 3
            for cfg in CONFIGS:
                y, zz, dx, dw = torch.empty_like(dy), torch.empty_like(z), torch.empty_like(x), torch.empty_like(w)
                outs = []
                for op in range(3):
                    try:
                        mb.mlp_linear_debug_set_plan(layer.h, op, cfg, split)
                    except MlpChainError:
                        # x^T dz has no short tiles, and one configuration of its own
                        assert cfg < 2 if op == 2 else cfg == 7
                        outs.append(None)
                        continue
                    if op == 0:
                        layer.forward(x, w, y, bias=b, residual=dy, z=zz)
                        outs.append((y, zz))
                    elif op == 1:
                        layer.backward(dy, None, w, dx=dx, z=z)
                        outs.append((dx,))
                    else:
                        layer.backward(dy, x, None, dw=dw, z=z)
                        outs.append((dw,))
                for op, got in enumerate(outs):
                    if got is None:
                        continue
                    seen[op] = seen[op] or got
                    assert all(torch.equal(p, q) for p, q in zip(seen[op], got)), (split, cfg, op)
        for op in range(3):
            mb.mlp_linear_debug_set_plan(layer.h, op, -1, 0)
        # the gradient's two products in one launch
        for cfg in CONFIGS:
            if cfg in (0, 7):
                with pytest.raises(MlpChainError, match="no tile configuration"):
                    mb.mlp_linear_debug_set_plan(layer.h, 3, cfg, 1)
                continue
            for sx, sw in ((1, 1), (2, 1), (1, 2), (4, 1), (1, 4)):
                mb.mlp_linear_debug_set_plan(layer.h, 3, cfg, sx)
                mb.mlp_linear_debug_set_plan(layer.h, 4, cfg, sw)
                dx, dw = torch.empty_like(x), torch.empty_like(w)
                layer.backward(dy, x, w, dx=dx, dw=dw, z=z)
                assert torch.equal(dx, results[sx][1][0]), (cfg, sx, sw)
                assert torch.equal(dw, results[sw][2][0]), (cfg, sx, sw)
        mb.mlp_linear_debug_set_plan(layer.h, 3, -1, 0)


@pytest.mark.parametrize("cfg,rows,K,N", [(0, 1100, 200, 600), (2, 2200, 328, 2200), (6, 2200, 200, 2200), (5, 2200, 200, 4200)])
def test_whole_tiles_beside_split_ones(cfg, rows, K, N):
    """More tiles than the chip has CUs: the first rounds are computed whole, the rest in parts."""
    c = linear_case(rows, K, N, "none", "f16", 10)
    y, y1 = torch.empty_like(c["dy"]), torch.empty_like(c["dy"])
    with MlpLinear(rows, K, N, "none", "f16") as layer:
        mb.mlp_linear_debug_set_plan(layer.h, 0, cfg, 1)
        layer.forward(c["x"], c["w"], y1, bias=c["bias"], residual=c["res"])
        mb.mlp_linear_debug_set_plan(layer.h, 0, cfg, 3)
        layer.forward(c["x"], c["w"], y, bias=c["bias"], residual=c["res"])
    x, w = c["x"].double(), c["w"].double()
    ref = torch.mm(x, w) + c["bias"].double() + c["res"].double()
    tol = (K / 32 + 64) * E32 * (torch.mm(x.abs(), w.abs()) + c["bias"].double().abs()) + 2.0 ** -20 * ref.abs()
    close(y, ref, rounded(ref, "f16") + tol, "split")
    close(y1, ref, rounded(ref, "f16") + tol, "whole")


@pytest.mark.parametrize("cfg,rows,K,N,sx,sw", [(1, 2200, 1104, 600, 3, 1), (6, 2200, 2200, 2312, 1, 3), (2, 1000, 2600, 2200, 2, 2)])
def test_both_products_of_more_tiles_than_cus(cfg, rows, K, N, sx, sw):
    """Whole and split tiles of both products of the gradient in one launch."""
    c = linear_case(rows, K, N, "none", "f16", 11)
    x, w, dy = c["x"], c["w"], c["dy"]
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    with MlpLinear(rows, K, N, "none", "f16") as layer:
        mb.mlp_linear_debug_set_plan(layer.h, 3, cfg, sx)
        mb.mlp_linear_debug_set_plan(layer.h, 4, cfg, sw)
        layer.backward(dy, x, w, dx=dx, dw=dw)
    for got, p, q in ((dx, dy.double(), w.double().t()), (dw, x.double().t(), dy.double())):
        ref = torch.mm(p, q)
        tol = (p.shape[1] / 32 + 64) * E32 * torch.mm(p.abs(), q.abs())
        close(got, ref, rounded(ref, "f16") + tol, "both")


@pytest.mark.parametrize("rows,act", [(1, "none"), (128, "swiglu"), (129, "none"), (300, "gelu_tanh"), (2500, "swiglu")])
def test_bias_gradient_does_not_depend_on_the_other_outputs(rows, act):
    """The column sums alone and in the launch of both products: the same bits."""
    c = linear_case(rows, 72, 1032, act, "bf16", 12)
    x, w, dy, z = c["x"], c["w"], c["dy"], c["z"]
    db = [torch.full_like(c["bias"], 7.0) for _ in range(3)]
    with MlpLinear(rows, 72, 1032, act, "bf16") as layer:
        layer.backward(dy, x, w, dx=torch.empty_like(x), dw=torch.empty_like(w), db=db[0], z=z)
        layer.backward(dy, None, None, db=db[1], z=z)
        layer.backward(dy, x, None, dw=torch.empty_like(w), db=db[2], z=z)
    assert torch.equal(db[0], db[1]) and torch.equal(db[0], db[2])


def test_forward_only_handles():
    c = linear_case(20, 264, 136, "gelu_tanh", "f16", 12)
    y, y2 = torch.empty_like(c["dy"]), torch.empty_like(c["dy"])
    x, w, b, dy, _ = norm_case(8, 264, "f16", 13)
    n, n2 = torch.empty_like(x), torch.empty_like(x)
    s = torch.ones(8, device="cuda")
    with MlpLinear(20, 264, 136, "gelu_tanh") as full, MlpLinear(20, 264, 136, "gelu_tanh", grad=False) as lin, \
            MlpNorm(264) as nfull, MlpNorm(264, grad=False) as norm:
        full.forward(c["x"], c["w"], y, bias=c["bias"])
        lin.forward(c["x"], c["w"], y2, bias=c["bias"])
        nfull.forward(x, w, b, n)
        norm.forward(x, w, b, n2)
        assert torch.equal(y, y2) and torch.equal(n, n2)
        with pytest.raises(MlpChainError, match="without its gradient"):
            lin.backward(c["dy"], c["x"], c["w"], dx=torch.empty_like(c["x"]), z=c["z"])
        with pytest.raises(MlpChainError, match="without its gradient"):
            norm.backward(dy, x, w, s, s, n)


def test_linear_outputs_left_out():
    c = linear_case(70, 264, 136, "gelu_tanh", "f16", 5)
    dx, dw, db = torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["bias"])
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    with MlpLinear(100, 264, 136, "gelu_tanh", "f16") as layer:
        layer.backward(c["dy"], c["x"], c["w"], dx=dx, dw=dw, db=db, z=c["z"])
        layer.backward(c["dy"], None, c["w"], dx=dx2, z=c["z"])
        layer.backward(c["dy"], c["x"], None, dw=dw2, z=c["z"])
        layer.backward(c["dy"], None, None, db=db2, z=c["z"])
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_linear_offsets_past_32_bits():
    """Rows 2^23 elements apart: byte offsets past 2^32 in every operand and output."""
    rows, K, N, ld = 300, 136, 136, 1 << 23
    c = linear_case(rows, K, N, "none", "f16", 6)
    base = torch.empty(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)
    y, y2 = torch.empty_like(c["res"]), base[:, 1024:1024 + N]
    far = base[:, :K]
    far.copy_(c["x"])
    dw, dw2, dx, dx2 = torch.empty_like(c["w"]), torch.empty_like(c["w"]), torch.empty_like(c["x"]), base[:, 2048:2048 + K]
    with MlpLinear(rows, K, N, "none", "f16") as layer:
        layer.forward(c["x"], c["w"], y, residual=c["res"])
        layer.forward(far, c["w"], y2, residual=c["res"])
        layer.backward(c["dy"], c["x"], c["w"], dx=dx, dw=dw)
        layer.backward(c["dy"], far, c["w"], dx=dx2, dw=dw2)
    assert torch.equal(y, y2) and torch.equal(dw, dw2) and torch.equal(dx, dx2)


# ------------------------------------------------------- calls, streams, graphs

def test_zero_rows():
    e = lambda n: torch.empty((0, n), dtype=torch.float16, device="cuda")  # noqa: E731
    w, b = torch.ones((64, 48), dtype=torch.float16, device="cuda"), torch.ones(48, dtype=torch.float16, device="cuda")
    with MlpNorm(64) as norm, MlpLinear(4, 64, 24, "swiglu") as lin:
        s = torch.empty(0, device="cuda")
        g = torch.ones(64, dtype=torch.float16, device="cuda")
        norm.forward(e(64), g, g, e(64), s, s)
        dg, db = torch.ones_like(g), torch.ones_like(g)
        norm.backward(e(64), e(64), g, s, s, e(64), dg, db)
        lin.forward(e(64), w, e(24), bias=b, residual=e(24), z=e(48))
        dw, dbias = torch.ones_like(w), torch.ones_like(b)
        lin.backward(e(24), e(64), w, dx=e(64), dw=dw, db=dbias, z=e(48))
    for t in (dg, db, dw, dbias):
        assert torch.equal(t, torch.zeros_like(t))


def test_fewer_rows_than_the_handle_holds():
    """One handle serves any row count up to its own, in any order, with the bits a handle of that size gives."""
    c = linear_case(600, 520, 264, "gelu_tanh", "f16", 7)
    with MlpLinear(600, 520, 264, "gelu_tanh") as big:
        for rows in (600, 1, 77, 16, 300):
            outs = []
            with MlpLinear(rows, 520, 264, "gelu_tanh") as own:
                for layer in (big, own):
                    x, dy, z = c["x"][:rows], c["dy"][:rows], c["z"][:rows]
                    y, dx, dw, db = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(c["w"]), torch.empty_like(c["bias"])
                    layer.forward(x, c["w"], y, bias=c["bias"])
                    layer.backward(dy, x, c["w"], dx=dx, dw=dw, db=db, z=z)
                    outs.append((y, dx, dw, db))
            assert all(torch.equal(a, b) for a, b in zip(*outs)), rows
        with pytest.raises(MlpChainError, match="rows"):
            y = torch.empty((601, 264), dtype=torch.float16, device="cuda")
            big.forward(torch.empty((601, 520), dtype=torch.float16, device="cuda"), c["w"], y)


def block_params(H, I, act, dtype, seed=41):
    n, dt = gen(seed), DT[dtype]
    gI = I * (2 if act == "swiglu" else 1)
    return {"weight": (1 + 0.1 * n(H)).to(dt), "bias": (0.1 * n(H)).to(dt), "w1": (n(H, gI) / math.sqrt(H)).to(dt),
            "b1": (0.1 * n(gI)).to(dt), "w2": (n(I, H) / math.sqrt(I)).to(dt), "b2": (0.1 * n(H)).to(dt)}


@pytest.mark.parametrize("rows,H,I,act,dtype", [(1, 512, 2048, "gelu_tanh", "f16"), (64, 512, 2048, "gelu_tanh", "f16"),
                                                (130, 520, 264, "swiglu", "bf16"), (33, 264, 136, "none", "f16")])
def test_block_forward_and_backward(rows, H, I, act, dtype):
    """The whole block and its gradients against 64-bit autograd of the definition: relative 2-norms within four
    roundings (the block rounds norm, inner activation, z and each of their gradients)."""
    p = block_params(H, I, act, dtype)
    n = gen(42)
    x, dy = n(rows, H).to(DT[dtype]), (0.1 * n(rows, H)).to(DT[dtype])
    with MlpBlock(rows, H, I, act, dtype, EPS) as block:
        y, saved = block.forward(x, p, save=True)
        assert torch.equal(block.forward(x, p), y)
        dx, grads = block.backward(dy, p, saved)
        torch.cuda.synchronize()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    xd = x.double().requires_grad_()
    h = torch.mm(norm_ref(xd, q["weight"], q["bias"])[0], q["w1"]) + q["b1"]
    ref = xd + torch.mm(act_ref(h, act, I), q["w2"]) + q["b2"]
    ref.backward(dy.double())
    for name, got, want in [("y", y, ref.detach()), ("dx", dx, xd.grad)] + [(k, grads[k], q[k].grad) for k in p]:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 4 * U[dtype], (name, rel)


def test_same_bits_again():
    c = linear_case(300, 2056, 264, "swiglu", "bf16", 51)
    x, w, b, dy, dr = norm_case(900, 2048, "bf16", 52)
    _, mean, rstd, _ = norm_ref(x, w, b)
    runs = []
    with MlpLinear(300, 2056, 264, "swiglu", "bf16") as lin, MlpNorm(2048, "bf16", EPS) as norm:
        for _ in range(3):
            y, dx, dw, db = torch.empty_like(c["dy"]), torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["bias"])
            lin.forward(c["x"], c["w"], y, bias=c["bias"])
            lin.backward(c["dy"], c["x"], c["w"], dx=dx, dw=dw, db=db, z=c["z"])
            nx, nw, nb = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
            norm.backward(dy, x, w, mean.float(), rstd.float(), nx, nw, nb, dres=dr)
            runs.append((y, dx, dw, db, nx, nw, nb))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_side_stream():
    """Work is ordered on the stream it is given: inputs produced there late are the ones that are read."""
    c = linear_case(64, 2048, 512, "gelu_tanh", "f16", 61)
    ref = torch.empty_like(c["dy"])
    with MlpLinear(64, 2048, 512, "gelu_tanh") as layer:
        layer.forward(c["x"], c["w"], ref, bias=c["bias"])
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        x, y = torch.zeros_like(c["x"]), torch.zeros_like(ref)
        torch.cuda.synchronize()
        big = torch.ones((4096, 4096), device="cuda")
        with torch.cuda.stream(s):
            for _ in range(4):
                big = torch.mm(big, big) * 1e-4
            x.copy_(c["x"])
            layer.forward(x, c["w"], y, bias=c["bias"])
        s.synchronize()
        assert torch.equal(y, ref)
        y.zero_()
        torch.cuda.synchronize()
        layer.forward(x, c["w"], y, bias=c["bias"], stream=s)
        s.synchronize()
        assert torch.equal(y, ref)


def test_graph_replays():
    """Forward and backward of the block's operators captured once, replayed with new inputs and eager work between."""
    rows, H, I = 48, 512, 2048
    p = block_params(H, I, "gelu_tanh", "f16")
    x = torch.zeros((rows, H), dtype=torch.float16, device="cuda")
    dy = torch.zeros_like(x)
    with MlpBlock(rows, H, I, "gelu_tanh", "f16", EPS) as block:
        def step():
            y, saved = block.forward(x, p, save=True)
            dx, grads = block.backward(dy, p, saved)
            return [y, dx] + [grads[k] for k in sorted(grads)]
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for i in range(4):
            n = gen(70 + i)
            x.copy_(n(rows, H))
            dy.copy_(0.1 * n(rows, H))
            want = [t.clone() for t in step()]
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


def test_refusals_of_tensors():
    h = torch.empty((4, 64), dtype=torch.float16, device="cuda")
    w = torch.empty((64, 32), dtype=torch.float16, device="cuda")
    out = torch.empty((4, 32), dtype=torch.float16, device="cuda")
    v = torch.empty(64, dtype=torch.float16, device="cuda")
    with MlpLinear(4, 64, 32, "gelu_tanh") as lin, MlpNorm(64) as norm:
        for bad in (h[:, :56], h.bfloat16(), h.t().contiguous().t(), h.cpu(), torch.empty((5, 64), dtype=torch.float16, device="cuda")):
            with pytest.raises((ValueError, MlpChainError)):
                lin.forward(bad, w, out)
            if bad.shape[0] == 4:
                with pytest.raises((ValueError, MlpChainError)):
                    norm.forward(bad, v, v, h)
        odd = torch.empty(4 * 64 + 8, dtype=torch.float16, device="cuda")[1:257].view(4, 64)
        with pytest.raises(MlpChainError, match="16-byte"):
            lin.forward(odd, w, out)
        with pytest.raises(MlpChainError, match="multiple of 8"):
            lin.forward(torch.empty((4, 68), dtype=torch.float16, device="cuda")[:, :64], w, out)
        with pytest.raises(MlpChainError, match="z must be"):
            lin.backward(out, h, w, dx=torch.empty_like(h))
        with pytest.raises(MlpChainError, match="w must be"):
            lin.backward(out, h, None, dx=torch.empty_like(h), z=out)
        with pytest.raises(MlpChainError, match="x must be"):
            lin.backward(out, None, w, dw=torch.empty_like(w), z=out)
        with pytest.raises(MlpChainError, match="mean and rstd"):
            norm.backward(h, h, v, None, None, torch.empty_like(h))
        with pytest.raises(ValueError):
            norm.forward(h, v, v, torch.empty_like(h), torch.empty(4, dtype=torch.float16, device="cuda"))
        with pytest.raises(ValueError):
            norm.forward(h, v[:32], v, torch.empty_like(h))
