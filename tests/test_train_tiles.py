"""The rows of the cross entropy's tall tiles, on the host (tests/native/train_tiles_selftest.cpp)."""
import os
import subprocess

import pytest

from consumer_gemm_chain_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tall_tiles_take_every_row_once(tmp_path):
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "train_tiles_selftest")
    cmd = [b.hipcc(), "-x", "hip", f"--offload-arch={b.ARCH}", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{b.CSRC}", os.path.join(ROOT, "tests", "native", "train_tiles_selftest.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout
