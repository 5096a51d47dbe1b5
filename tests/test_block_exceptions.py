"""No C++ exception leaves the library's C interface: errors are reported with the process out of host memory."""
import os
import shutil
import subprocess

import pytest

from consumer_gemm_chain_amd import mlp_chain as mc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_errors_without_host_memory(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = str(tmp_path / "block_throw_selftest")
    libdir = os.path.dirname(mc.LIB_PATH)
    r = subprocess.run(["g++", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}",
                        os.path.join(ROOT, "tests", "native", "block_throw_selftest.cpp"), "-o", exe, mc.LIB_PATH,
                        f"-Wl,-rpath,{libdir}", "-Wl,--allow-shlib-undefined"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "0 failures" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])
