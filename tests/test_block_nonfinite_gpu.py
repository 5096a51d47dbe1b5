"""NaN and infinity in the block operators' operands: they reach the outputs that the formulas make depend on them, and
no others.  The reference is the formula in 64 bits on the CPU; the other outputs are held to a rounding of the type
and the fp32 arithmetic's error, which is far below the half roundoff added here."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLinear, MlpNorm  # noqa: E402
from consumer_gemm_chain_amd import mlp_block as mb  # noqa: E402
from tests.test_block_gpu import DT, TINY, U, EPS, act_ref, linear_case, norm_case  # noqa: E402

INF, NAN = float("inf"), float("nan")


def same_class(got, ref, dtype, scale, what):
    """Non-finite in the same places, and elsewhere within a rounding and a half of `ref`, or of sums of size `scale`."""
    got, ref = got.double().cpu(), ref.double().cpu()
    assert torch.equal(got.isfinite(), ref.isfinite()), (what, (got.isfinite() != ref.isfinite()).nonzero()[:4].tolist())
    fine = ref.isfinite()
    off = (got - ref).abs()[fine]
    assert (off <= 1.5 * U[dtype] * ref.abs()[fine] + 2.0 ** -14 * scale + TINY[dtype]).all(), (what, float(off.max()))


def cpu(t):
    return None if t is None else t.double().cpu()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,H", [(6, 24), (6, 333), (40, 512), (6, 8192), (6, 9001), (5, 20000), (5, 5)])
@pytest.mark.parametrize("where", ["x", "dy", "dres", "weight", "last x", "last dy"])
def test_norm_gradient(where, rows, H, dtype):
    x, w, b, dy, dr = norm_case(rows, H, dtype, 5)
    if where == "weight":
        w[H // 2] = NAN
    else:
        t = {"x": x, "dy": dy, "dres": dr}[where.split()[-1]]
        r = rows - 1 if where.startswith("last") else 1
        t[r, H - 1] = NAN
        t[r - 1, 0] = INF
        t[r - 1, H // 2] = -INF
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    with MlpNorm(H, dtype, EPS) as layer:
        layer.forward(x, w, b, y, mean, rstd)
        layer.backward(dy, x, w, mean, rstd, dx, dw, db, dres=dr)
        torch.cuda.synchronize()
    xd, wd, bd, dyd, drd, m, rs = (cpu(t) for t in (x, w, b, dy, dr, mean, rstd))
    xhat = (xd - m[:, None]) * rs[:, None]
    g = dyd * wd
    ref = rs[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) + drd
    same_class(y, xhat * wd + bd, dtype, 4, "y")
    same_class(dx, ref, dtype, 1, "dx")
    same_class(dw, (dyd * xhat).sum(0), dtype, 4, "dweight")
    same_class(db, dyd.sum(0), dtype, 4, "dbias")


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows,split", [(20, 0), (300, 0), (300, 3)])
def test_linear_forward(rows, split, act):
    K, N, dtype = 328, 264, "f16"
    c = linear_case(rows, K, N, act, dtype, 7)
    x, w, bias, res = c["x"], c["w"], c["bias"], c["res"]
    x[1, 5], x[3, K - 1], x[rows - 1, 0] = NAN, INF, -INF
    w[17, 9], w[100, N - 1] = NAN, INF
    bias[40], res[2, 11], res[4, 200] = -INF, NAN, INF
    y, z = torch.empty_like(c["dy"]), torch.empty_like(c["z"])
    with MlpLinear(rows, K, N, act, dtype) as layer:
        if split:
            mb.mlp_linear_debug_set_plan(layer.h, 0, 2, split)
        layer.forward(x, w, y, bias=bias, residual=res, z=z)
        torch.cuda.synchronize()
    h = torch.mm(cpu(x), cpu(w)) + cpu(bias)
    same_class(z, h, dtype, 8, "z")
    same_class(y, act_ref(h, act, N) + cpu(res), dtype, 32, "y")


def gelu_slope(z):
    """The gelu's derivative with its limits, 1 and 0, at the infinities."""
    t = z.clamp(-40, 40)
    s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))
    return s + t * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * t * t)


@pytest.mark.parametrize("act", ["none", "gelu_tanh", "swiglu"])
@pytest.mark.parametrize("rows", [20, 300])
@pytest.mark.parametrize("joint", [True, False])
def test_linear_gradient(rows, act, joint):
    """dz, and with it every product, at infinities and NaN in z and dy; dx sees w's, dw sees x's."""
    K, N, dtype = 328, 264, "f16"
    c = linear_case(rows, K, N, act, dtype, 8)
    x, w, dy, z = c["x"], c["w"], c["dy"], c["z"]
    z[1, 5], z[2, 6], z[3, 7], z[rows - 1, c["gN"] - 1] = NAN, INF, -INF, INF
    dy[4, 50], dy[6, 60] = NAN, INF
    x[7, 5], x[9, K - 1] = NAN, -INF
    w[17, 9], w[K - 1, N - 1] = NAN, INF
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(c["bias"])
    with MlpLinear(rows, K, N, act, dtype) as layer:
        if joint:
            layer.backward(dy, x, w, dx=dx, dw=dw, db=db, z=z)
        else:
            layer.backward(dy, None, w, dx=dx, z=z)
            layer.backward(dy, x, None, dw=dw, z=z)
            layer.backward(dy, None, None, db=db, z=z)
        torch.cuda.synchronize()
    d, zd = cpu(dy), cpu(z)
    if act == "gelu_tanh":
        d = d * gelu_slope(zd)
    elif act == "swiglu":
        g, u = zd[:, :N], zd[:, N:]
        s = torch.sigmoid(g)
        d = torch.cat([d * u * (s + g * s * (1 - s)), d * (g * s)], 1)
    rounded = d.half().double()
    same_class(db, d.sum(0), dtype, 64, "db")
    same_class(dx, torch.mm(rounded, cpu(w).t()), dtype, 32, "dx")
    same_class(dw, torch.mm(cpu(x).t(), rounded), dtype, 64, "dw")
