"""Calls on tall tiles whose rows are all left out, on the host: no division by their number
(tests/native/train_no_rows_selftest.cpp, under the undefined-behaviour sanitizer)."""
import os
import subprocess

import pytest

from consumer_gemm_chain_amd import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("opt", ["-O0", "-O2"])
def test_no_rows_have_no_tall_tiles(tmp_path, opt):
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "train_no_rows_selftest")
    san = ["-Xarch_host", "-fsanitize=undefined,float-divide-by-zero", "-Xarch_host", "-fno-sanitize-recover=all"]
    cmd = [b.hipcc(), "-x", "hip", f"--offload-arch={b.ARCH}", opt, "-g", "-std=c++17", *san,
           f"-I{os.path.join(ROOT, 'include')}", f"-I{b.CSRC}", os.path.join(ROOT, "tests", "native", "train_no_rows_selftest.cpp"),
           "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "0 failures" in r.stdout and "runtime error" not in r.stderr, (r.stdout, r.stderr[-3000:])
