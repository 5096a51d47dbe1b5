"""AdamW at the border of what fp32 holds, against the formula in 64 bits."""
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
