"""Optimizers whose tensors share memory are refused when they are made: nothing has run on them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW  # noqa: E402


def test_shared_states_are_refused():
    flat = torch.randn(1 << 12, device="cuda").half()
    w = list(flat.split([2048, 1024, 1024]))
    one = torch.zeros(4096, device="cuda")
    apart, other = (list(torch.zeros(4096, device="cuda").split([2048, 1024, 1024])) for _ in range(2))
    with MlpAdamW(w, "f16", m=apart, v=other) as opt:                                   # views of one buffer are apart
        opt.step([torch.ones_like(t) for t in w], 1e-3)
        torch.cuda.synchronize()
    for bad in ({"m": [one[:t.numel()] for t in w]}, {"m": apart, "v": apart}, {"master": apart, "m": apart},
                {"m": [one[:2048], one[2047:3071], one[3072:]]}):
        with pytest.raises(ValueError, match="share memory"):
            MlpAdamW(w, "f16", **bad)
    with pytest.raises(ValueError, match="share memory"):
        MlpAdamW([flat[:100], flat[99:200]], "f16")
    scales = [torch.ones(8, device="cuda")] * 2
    with pytest.raises(ValueError, match="share memory"):
        MlpAdamW([w[0], w[1]], "f16", 8, m_scale=[scales[0], scales[0][:4]])
