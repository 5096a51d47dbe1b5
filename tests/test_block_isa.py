"""The compiled gfx950 code of the block operators' kernels (no GPU needed):
no packed fp32 arithmetic anywhere, no register spills in the linear layer's
kernels, operand DMA in the scalar-base form, no scratch in a K loop."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from consumer_gemm_chain_amd import build as b


def _compile(job):
    src, defs, out = job
    cmd = [b.hipcc(), "-x", "hip", *b.FLAGS, *defs, "--cuda-device-only", "-S", os.path.join(b.CSRC, src), "-o", str(out)]
    subprocess.run(cmd, check=True, stderr=subprocess.DEVNULL)
    return out.read_text()


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("block_isa")
    jobs = {f"linear{c}": (b.LINEAR_KERNELS, [f"-DMLPC_LIN={c}"], d / f"linear{c}.s")
            for c in range(b.num_configs("linear_configs.h"))}
    for src in b.BLOCK_SOURCES:
        if src.endswith(".hip"):
            jobs[src] = (src, [], d / (src + ".s"))
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        return dict(zip(jobs, ex.map(_compile, jobs.values())))


def _kernels(text):
    for m in re.finditer(r"- \.agpr_count:.*?\.wavefront_size:", text, flags=re.S):
        field = lambda k: re.search(rf"\.{k}:\s+(\S+)", m.group(0)).group(1)  # noqa: E731
        yield field("name"), int(field("vgpr_spill_count")), int(field("sgpr_spill_count"))


def test_no_packed_fp32_arithmetic(asm):
    for name, text in asm.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), name


def test_register_spills(asm):
    """None, but a few values of the norm gradient for rows past 12288 (two
    chunks per thread in the registers of 16 waves)."""
    for name, text in asm.items():
        kernels = list(_kernels(text))
        assert kernels, name
        for kernel, spill, sspill in kernels:
            wide = re.search(r"norm_backward_kernelILi\dELi1024ELi2E", kernel)
            assert spill <= (16 if wide else 0), (name, kernel, spill)
            assert sspill == 0, (name, kernel, sspill)


def test_linear_kernels_stream_in_the_scalar_base_form(asm):
    for name, text in asm.items():
        if not name.startswith("linear") or name.endswith(".hip"):
            continue
        bodies = re.findall(r"^(_ZN4mlpc\d+linear_(?:both_)?kernel\w*):(.*?)\.Lfunc_end", text, flags=re.M | re.S)
        assert len(bodies) >= 2, name
        for kernel, body in bodies:
            assert re.search(r"global_load_lds_dwordx4 v\d+, s\[\d+:\d+\]", body), kernel
            assert "scratch_" not in body, kernel
            assert "v_mfma_f32_16x16x32" in body, kernel
