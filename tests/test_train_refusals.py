"""Arguments of the training step's operators that fp32 cannot hold are refused, with a message (no GPU needed)."""
import os
import subprocess

import pytest

from consumer_gemm_chain_amd import build as b
from consumer_gemm_chain_amd import mlp_chain as mc
from consumer_gemm_chain_amd import mlp_train as mt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [5e-324, 1e-50, 1e-45, 1e-39, 2.0 ** -126 * (1 - 2.0 ** -24)])
def test_an_eps_below_the_smallest_normal_number_is_refused(eps, bits):
    """Its reciprocal is infinite in fp32: an element without a gradient would become NaN."""
    with pytest.raises(mc.MlpChainError, match="eps"):
        mt.mlp_adamw_create(0, bits, 0.9, 0.99, eps, 0)


def test_an_unscale_that_fp32_cannot_hold_is_refused(tmp_path):
    """Its scale would be infinite, which leaves steps out that have finite gradients, or zero, or a subnormal with few bits
    (tests/native/train_refusals_selftest.cpp, on a stand-in for the HIP runtime)."""
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "train_refusals_selftest")
    cmd = [b.hipcc(), "-x", "hip", f"--offload-arch={b.ARCH}", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{b.CSRC}", os.path.join(b.CSRC, "train_api.cpp"),
           os.path.join(ROOT, "tests", "native", "train_refusals_selftest.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "0 failures" in r.stdout, (r.stdout, r.stderr[-3000:])
