"""Arguments of the training step's operators that fp32 cannot hold are refused, with a message (no GPU needed)."""
import pytest

from consumer_gemm_chain_amd import mlp_chain as mc
from consumer_gemm_chain_amd import mlp_train as mt


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [5e-324, 1e-50, 1e-45, 1e-39, 2.0 ** -126 * (1 - 2.0 ** -24)])
def test_an_eps_below_the_smallest_normal_number_is_refused(eps, bits):
    """Its reciprocal is infinite in fp32: an element without a gradient would become NaN."""
    with pytest.raises(mc.MlpChainError, match="eps"):
        mt.mlp_adamw_create(0, bits, 0.9, 0.99, eps, 0)
