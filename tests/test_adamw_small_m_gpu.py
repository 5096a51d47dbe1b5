"""AdamW's m in e4m3 far below its block's largest.  Below the normal numbers, 2^-6 of the scale, codes are 2^-9 apart, and a step
without a gradient takes (1 - beta1) k of code k away: less than half a code for k <= 4 and a beta1 of 0.9.  Rounded to nearest,
such an m would stay for good, beside a v that falls to its smallest number, and its weight would be moved by a part of lr
at every step.  Where rounding to nearest would give the old code again, these are rounded up or down by chance."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW  # noqa: E402
from tests.test_optim_gpu import E4, block_scale, mix, per_element  # noqa: E402


def m_codes(m, scale, old, t, seed):
    """e4m3 values of m in units of its block's scale, `old` what m was before the step: to nearest, but by chance, with the
    random bits that the pair's other v is rounded with, where that is the old value, below 2^-6 and not zero."""
    n = m.numel()
    y = m / per_element(scale, n)
    near = y.to(E4).float()
    k = torch.floor(y.abs().double() * 512 * 2.0 ** 20) / 2.0 ** 20        # (cut after 23 bits of 2^-6 + y)
    same = (y.abs() < 2.0 ** -6) & (y != 0) & (near != 0) & (near.abs().double() == old.abs().double() / per_element(scale, n).double())
    place = torch.arange(n, device=m.device)
    key = mix(torch.tensor((int(mix(torch.tensor((t + seed) & 0xFFFFFFFF)))) & 0xFFFFFFFF))
    r = mix(((place >> 1) + int(key)) & 0xFFFFFFFF)
    u = torch.where(place % 2 == 0, r >> 16, r & 0xFFFF).double() / 65536
    return torch.where(same, (torch.floor(k + u) / 512 * torch.sign(y.double())).float(), near), same


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("b1", [0.9, 0.5, 0.9375])
def test_codes_of_small_m(b1, dtype):
    """Bit for bit: numbers of all sizes in a block, two thirds of them without a gradient, and a ragged end."""
    n = 20011
    gen = torch.Generator("cuda").manual_seed(1)
    sign = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    m0 = sign * torch.exp2(-22 * torch.rand(n, generator=gen, device="cuda"))
    m0[torch.rand(n, generator=gen, device="cuda") < 0.05] = 0
    scale = block_scale(m0, 8)
    m = (m0 / per_element(scale, n)).to(E4)
    old = m.float() * per_element(scale, n)
    dt = torch.float16 if dtype == "f16" else torch.bfloat16
    g = (old * torch.randn(n, generator=gen, device="cuda")).to(dt)
    g[torch.rand(n, generator=gen, device="cuda") < 0.66] = 0
    want_m = old * b1 + g.float() * (1 - b1)
    want_scale = block_scale(want_m, 8)
    w = torch.zeros(n, device="cuda").to(dt)
    with MlpAdamW([w], dtype, 8, beta1=b1, seed=77, m=[m], m_scale=[scale]) as opt:
        opt.step([g], 1e-3)
        torch.cuda.synchronize()
    want, same = m_codes(want_m, want_scale, old, 1, 77)
    assert b1 == 0.5 or int(same.sum()) > 300
    assert torch.equal(scale, want_scale) and torch.equal(m.float(), want)


def test_small_m_falls_as_it_should():
    """The mean of codes 1 to 4 after k steps without a gradient is 0.9^k of them, beside an element that keeps the scale: codes
    lie in 0..4, so the mean of n of them has a sigma of at most 2 / sqrt(n); random bits are 16: at most 2^-16 a step."""
    n, steps = 1 << 18, 10
    first = torch.arange(n, device="cuda") % 256 == 0
    k0 = (torch.arange(n, device="cuda") % 4 + 1).float()
    m = torch.where(first, 384.0, k0 / 512).to(E4)
    scale = torch.ones(n // 256, device="cuda")
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.where(first, 384.0, 0.0).bfloat16()
    with MlpAdamW([w], "bf16", 8, beta1=0.9, m=[m], m_scale=[scale]) as opt:
        for k in range(1, steps + 1):
            opt.step([g], 0.0)
            torch.cuda.synchronize()
            assert (scale == 1).all() and (m.float()[first] == 384).all()
            code = (m.float() * 512)[~first].double()
            for j in (1, 2, 3, 4):
                got = code[k0[~first] == j]
                assert abs(float(got.mean()) - j * 0.9 ** k) <= 6 * 2 / math.sqrt(got.numel()) + k * 2.0 ** -16


@pytest.mark.parametrize("b1", [0.9, 0.95])
def test_weights_without_a_gradient_come_to_rest(b1):
    """Half of each block's weights lose their gradients after 50 steps; 550 steps later they do not move any more.  After 200 of
    these m is at most 8 codes in the mean (448 x 512 x 0.95^200), and each step takes 1 - beta1 of the mean: that any of the 4096
    is left after 350 more has a chance of at most 4096 x 8 x 0.95^350 = 5e-4."""
    n = 256 * 32
    gen = torch.Generator("cuda").manual_seed(1)
    master = torch.zeros(n, device="cuda")
    w = master.bfloat16()
    alive = torch.arange(n, device="cuda") % 2 == 0
    with MlpAdamW([w], "bf16", 8, beta1=b1, beta2=0.95, master=[master]) as opt:
        for k in range(650):
            g = torch.randn(n, generator=gen, device="cuda")
            if k >= 50:
                g = g * alive
            if k == 600:
                before = master.clone()
            opt.step([g.bfloat16()], 1e-3)
        torch.cuda.synchronize()
        assert (opt.m[0].float()[~alive] == 0).all()
        assert (opt.v[0].float()[~alive] > 0).all()
    assert torch.equal(master[~alive], before[~alive])
    assert (master[alive] != before[alive]).all()
