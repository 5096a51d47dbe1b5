"""The training step's handles on a stand-in for the HIP runtime (tests/native/train_runtime_selftest.cpp, whose
definitions take the place of the library's): workspaces, refusals, tables, errors and streams, under the host
sanitizers."""
import os
import subprocess

import pytest

from consumer_gemm_chain_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_train_handles_on_a_stand_in_runtime(tmp_path):
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not available")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all"]
    exe = str(tmp_path / "train_runtime_selftest")
    cmd = [b.hipcc(), "-x", "hip", f"--offload-arch={b.ARCH}", "-O1", "-g", "-std=c++17", *san,
           f"-I{os.path.join(ROOT, 'include')}", f"-I{b.CSRC}", os.path.join(b.CSRC, "train_api.cpp"),
           os.path.join(ROOT, "tests", "native", "train_runtime_selftest.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    # (leaks are not checked: the HIP runtime keeps allocations until exit)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600,
                       env={**os.environ, "ASAN_OPTIONS": "detect_leaks=0"})
    assert r.returncode == 0 and "0 failures" in r.stdout and "runtime error" not in r.stderr, (r.stdout, r.stderr[-3000:])
