"""AdamW at the border of what fp32 holds, against the formula in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW  # noqa: E402


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [2.0 ** -126, 2.0 ** -125, 1e-30, 2.0 ** -40, 2.0 ** -39])
def test_elements_without_a_gradient_stay_where_they_are(eps, bits):
    """m and v of zero change nothing, however small eps is; the others move by lr in a first step."""
    n = 3001
    gen = torch.Generator("cuda").manual_seed(1)
    g = torch.randn(n, generator=gen, device="cuda").bfloat16()
    g[::3] = 0
    master = torch.randn(n, generator=gen, device="cuda")
    before, w = master.clone(), master.bfloat16()
    with MlpAdamW([w], "bf16", bits, eps=eps, master=[master]) as opt:
        opt.step([g], 2.0 ** -7)
        torch.cuda.synchronize()
        assert (opt.m[0].float()[::3] == 0).all() and (opt.v[0].float()[::3] == 0).all()
    assert torch.equal(master[::3], before[::3])
    d = g.double()
    want = before.double() - torch.where(d != 0, 2.0 ** -7 * d / (d.abs() + eps), 0.0)
    # hardware root and reciprocal: 2^-20 of the change; then the weight's rounding
    assert ((master.double() - want).abs() <= 2.0 ** -27 + 2.0 ** -24 * want.abs()).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("decay", [1e-6, 1e-5, 1e-4, 1e-2, 0.75])
def test_a_small_decay_is_not_rounded_before_the_weight_takes_it(decay, bits):
    """Weights without a gradient, w (1 - d) by the formula: d and d w are within 2^-23 of themselves, and w is rounded once.
    A factor 1 - d that is rounded on its own is off by up to 2^-25, the same way at every step: of d = 1e-6 that is 3%.

    The mean decay of many weights shows it.  With a mantissa m in [1, 2) and D = d 2^23 the decay is D m ulps and its
    rounding e(D m), a sawtooth whose integral over m, taken around its middle, stays within 1 / (16 D).  Mantissas have the density
    1 / (m ln 2), so the mean of e / (D m) is at most 1 / (16 D) times the variation of f = 1 / (m^2 D ln 2) over the mantissas: f rises
    from 0 to f(1) and falls to 0, and the thousandth of a binade that is left out adds at most as much again, 4 f(1) in all.
    That is 1 / (4 ln 2 D^2); besides, six sigma of a mean of n roundings of at most half an ulp."""
    n, steps = 1 << 20, 3
    gen = torch.Generator("cuda").manual_seed(2)
    sign = torch.where(torch.arange(n, device="cuda") % 2 == 0, 1.0, -1.0)
    master = torch.exp2(torch.rand(n, generator=gen, device="cuda") * 0.999) * sign
    w, g = master.bfloat16(), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    with MlpAdamW([w], "bf16", bits, decay=1.0, master=[master]) as opt:
        for _ in range(steps):
            before = master.double()
            opt.step([g], decay)
            torch.cuda.synchronize()
            want = before * (1 - decay)
            assert ((master.double() - want).abs() <= (2.0 ** -24 + 2.0 ** -22 * decay) * before.abs()).all()
            assert torch.equal(w, master.bfloat16())
            mean = float(((before - master.double()) / before).mean()) / decay
            D = decay * 2.0 ** 23
            assert abs(mean - 1) <= 1 / (4 * math.log(2.0) * D * D) + 6 / (2 * D * n ** 0.5) + 2.0 ** -22
