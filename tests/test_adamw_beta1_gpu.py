"""AdamW's m in e4m3 with a beta1 near one.  Without a gradient a step leaves beta1 m.  Rounded to nearest that is m itself
where (1 - beta1) m is less than half a step of e4m3, 1/16 for an m of 1.125: from beta1 = 17/18 on such an m would never
fall, while v does.  Past 15/16 m is therefore rounded up or down by chance, with a mean of m."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW  # noqa: E402
from tests.test_optim_gpu import E4, Case, block_scale, mix, per_element, v_codes  # noqa: E402


def m_codes(m, scale, t, seed, number):
    """e4m3 values of m in units of its block's scale: floor(y / step + u) steps, u from the half of a pair's random bits that
    the other element's v is rounded with.  (A subnormal y is taken with 2^-6 added, cut after 23 bits of fraction.)"""
    n = m.numel()
    y = (m.abs() / per_element(scale, n)).double()
    place = torch.arange(n, device=m.device)
    key = mix(torch.tensor((int(mix(torch.tensor((t + seed) & 0xFFFFFFFF))) + 0x9E3779B9 * number) & 0xFFFFFFFF))
    r = mix(((place >> 1) + int(key)) & 0xFFFFFFFF)
    u = torch.where(place % 2 == 0, r >> 16, r & 0xFFFF).double() / 65536
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    y = torch.where(y < 2.0 ** -6, torch.floor((y + 2.0 ** -6) * 2.0 ** 29) / 2.0 ** 29 - 2.0 ** -6, y)
    return (torch.floor(y / step + u) * step * torch.sign(m.double())).float()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("b1", [0.9376, 0.95, 0.99, 0.9999])
def test_m_is_rounded_by_chance(b1, master, dtype):
    """Codes bit for bit, at several sizes and places, and everything else as with any beta1."""
    c = Case([1, 7, 256, 257, 0, 5000, 2048, 40], dtype, 8, master, shift=1, b1=b1)
    expected = c.expected(1e-3)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    for i, (ref, tol, m, v) in enumerate(expected):
        got = c.master[i] if master else c.w[i]
        u = 0.0 if master else torch.finfo(c.w[i].dtype).eps / 2
        assert ((got.double() - ref).abs() <= tol + u * ref.abs() + (0 if master else 2.0 ** -25)).all(), ("w", i)
        ms, vs = block_scale(m, 8), block_scale(v, 15)
        assert torch.equal(c.m_scale[i], ms) and torch.equal(c.v_scale[i], vs), ("scales", i)
        assert torch.equal(c.m[i].float(), m_codes(m, ms, int(c.t), c.seed, i)), ("m", i)
        assert torch.equal(c.v[i].float(), v_codes(v, vs, int(c.t), c.seed, i)), ("v", i)
    assert all(ok() for ok in c.checks), "written around a tensor"


@pytest.mark.parametrize("b1", [0.0, 0.5, 0.9, 0.9375])
def test_m_is_rounded_to_nearest_up_to_fifteen_sixteenths(b1):
    c = Case([1, 257, 5000], "bf16", 8, True, b1=b1)
    expected = c.expected(1e-3)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    c.check(expected)


@pytest.mark.parametrize("b1", [0.95, 0.99])
def test_m_falls_when_gradients_have_gone(b1):
    """The mean of m / (beta1^k m0) is 1.  A rounding by chance between neighbours a step apart has at most a quarter of the
    step's square as its variance, and a step of e4m3 is at most 1/8 of a normal number: after k steps the variance of the ratio
    is at most (1 + 2^-8)^k - 1.  Six sigma of a mean of n; random bits are 16, so a mean is off by 2^-16 of a step, 2^-19, at
    each rounding besides.  (m0 spans one binade, so no code is subnormal.)"""
    n, steps = 1 << 18, 20
    gen = torch.Generator("cuda").manual_seed(4)
    m0 = (1 + torch.rand(n, generator=gen, device="cuda")) * torch.where(torch.arange(n, device="cuda") % 3 == 0, -1.0, 1.0)
    scale = block_scale(m0, 8)
    m = (m0 / per_element(scale, n)).to(E4)
    m0 = m.float() * per_element(scale, n)
    w, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    with MlpAdamW([w], "bf16", 8, beta1=b1, m=[m], m_scale=[scale]) as opt:
        for _ in range(steps):
            opt.step([g], 0.0)
        torch.cuda.synchronize()
    ratio = (m.float() * per_element(scale, n) / m0).double() / b1 ** steps
    sigma = math.sqrt((1 + 2.0 ** -8) ** steps - 1)
    assert abs(float(ratio.mean()) - 1) <= 6 * sigma / math.sqrt(n) + steps * 2.0 ** -19


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_gradient_that_is_not_finite(bad):
    """Its element's m is NaN; the others of its block are what they would be."""
    c = Case([700], "bf16", 8, True, b1=0.95)
    c.grad[0][300] = bad
    (_, _, m, _), = c.expected(1e-3)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    assert c.m[0][300].float().isnan() and c.v[0][300].float().isnan()
    keep = torch.arange(700, device="cuda") != 300
    scale = block_scale(m, 8)
    want = m_codes(torch.where(keep, m, 0.0), scale, int(c.t), c.seed, 0)
    assert torch.equal(c.m_scale[0], scale) and torch.equal(c.m[0].float()[keep], want[keep])
