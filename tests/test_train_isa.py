"""The compiled gfx950 code of the training step's kernels (no GPU needed): no packed fp32 arithmetic, no register spills
or scratch, operand DMA in the scalar-base form and matrix instructions in the cross entropy's products."""
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
    d = tmp_path_factory.mktemp("train_isa")
    jobs = {f"loss{c}": (b.LOSS_KERNELS, [f"-DMLPC_LOSS={c}"], d / f"loss{c}.s")
            for c in range(b.num_configs("loss_configs.h"))}
    for src in b.TRAIN_SOURCES:
        if src.endswith(".hip"):
            jobs[src] = (src, [], d / (src + ".s"))
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        return dict(zip(jobs, ex.map(_compile, jobs.values())))


def test_no_packed_fp32_arithmetic(asm):
    for name, text in asm.items():
        assert not re.search(r"v_pk_(add|mul|fma)_f32", text), name


def test_no_register_spills(asm):
    for name, text in asm.items():
        kernels = re.findall(r"- \.agpr_count:.*?\.wavefront_size:", text, flags=re.S)
        assert kernels, name
        for k in kernels:
            field = lambda f: re.search(rf"\.{f}:\s+(\S+)", k).group(1)  # noqa: E731,B023
            for f in ("vgpr_spill_count", "sgpr_spill_count", "private_segment_fixed_size"):
                assert int(field(f)) == 0, (name, field("name"), f)


def test_products_stream_in_the_scalar_base_form(asm):
    for name, text in asm.items():
        if name.endswith(".hip"):
            continue
        bodies = re.findall(r"^(_ZN4mlpc\d+loss_(?:logits|products)_kernel\w*):(.*?)\.Lfunc_end", text, flags=re.M | re.S)
        assert len(bodies) == (4 if name == "loss0" else 6), name
        for kernel, body in bodies:
            assert re.search(r"global_load_lds_dwordx4 v\d+, s\[\d+:\d+\]", body), kernel
            assert "v_mfma_f32_16x16x32" in body, kernel


def test_kernel_arguments_fit(asm):
    """Tables of tensors travel as arguments: at most 4 KB."""
    for name, text in asm.items():
        for size in re.findall(r"\.kernarg_segment_size:\s+(\d+)", text):
            assert int(size) <= 4096, name
