"""Gradient norm and AdamW of one tensor whose elements and bytes pass 2^31, and of many tensors that take several tables."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW, MlpGradNorm  # noqa: E402
from tests.test_optim_gpu import block_scale, mix  # noqa: E402

N = (1 << 31) + 777
# looked at: the ends, and what lies around 2^31 and the places that 32-bit offsets in bytes would wrap to
PARTS = [slice(0, 2048), slice((1 << 29) - 1024, (1 << 29) + 1024), slice((1 << 30) - 1024, (1 << 30) + 1024),
         slice((1 << 31) - 1024, (1 << 31) + 512), slice((1 << 31) + 512, N)]


def test_the_norm_of_a_tensor_past_two_to_the_31():
    g = torch.full((N,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    g[-1] = 1000.0
    norm, scale = (torch.empty(1, device="cuda") for _ in range(2))
    with MlpGradNorm("bf16") as layer:
        layer.forward([g], norm, scale, max_norm=1.0)
        torch.cuda.synchronize()
    want = math.sqrt((N - 1) * 2.0 ** -20 + float(g[-1]) ** 2)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want and abs(float(scale) - 1 / want) <= 2.0 ** -23 / want


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_of_a_tensor_past_two_to_the_31(bits):
    """Zeros but in the parts that are looked at, where m, v, scales and codes are those of the formula at their places; every
    other element stays zero."""
    gen = torch.Generator("cuda").manual_seed(1)
    w, g = (torch.zeros(N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for s in PARTS:
        g[s] = torch.randn(s.stop - s.start, generator=gen, device="cuda").bfloat16()
    with MlpAdamW([w], "bf16", bits, seed=5) as opt:
        opt.step([g], 2.0 ** -7)
        torch.cuda.synchronize()
        m, v = opt.m[0], opt.v[0]
        for s in PARTS:
            f = g[s].float()
            want_m, want_v = f * (1 - 0.9), (f * f) * (1 - 0.999)
            d = f.double()
            want = -2.0 ** -7 * d / (d.abs() + 1e-8)
            assert ((w[s].double() - want).abs() <= 2.0 ** -7 * (2.0 ** -8 + 2.0 ** -20)).all()
            if bits == 32:
                assert torch.equal(m[s], want_m) and torch.equal(v[s], want_v)
                continue
            blocks = slice(s.start // 256, -(-s.stop // 256))
            ms, vs = block_scale(want_m, 8), block_scale(want_v, 15)
            assert torch.equal(opt.m_scale[0][blocks], ms) and torch.equal(opt.v_scale[0][blocks], vs)
            assert torch.equal(m[s].float(), (want_m / ms.repeat_interleave(256)[:len(f)]).to(torch.float8_e4m3fn).float())
            y = (want_v / vs.repeat_interleave(256)[:len(f)]).double()
            place = torch.arange(s.start, s.stop, device="cuda")
            key = int(mix(torch.tensor(int(mix(torch.tensor(1 + 5))))))
            r = mix(((place >> 1) + key) & 0xFFFFFFFF)
            u = torch.where(place % 2 == 0, r & 0xFFFF, r >> 16).double() / 65536
            step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -14))) - 2)
            y = torch.where(y < 2.0 ** -14, (y.float() + 2.0 ** -14).double() - 2.0 ** -14, y)
            q = torch.floor(y / step + u)
            assert torch.equal(v[s].float(), (torch.where((want_v > 0) & (q < 1), 1.0, q) * step).float())
        rest = torch.ones(N, dtype=torch.bool, device="cuda")
        for s in PARTS:
            rest[s] = False
        for t in (w, m, v):
            words = t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])
            for at in range(0, N, 1 << 28):
                part = slice(at, min(at + (1 << 28), N))
                assert not bool((words[part][rest[part]] != 0).any())


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_of_one_and_none(bits):
    """Several tables of single elements, with empty tensors at the tables' ends."""
    count = 48 * 3 + 1
    sizes = [0 if i % 48 in (0, 47) else 1 for i in range(count)]
    w = [torch.zeros(k, dtype=torch.float16, device="cuda") for k in sizes]
    g = [torch.full((k,), float(i + 1), device="cuda").half() for i, k in enumerate(sizes)]
    norm = torch.empty(1, device="cuda")
    with MlpAdamW(w, "f16", bits) as opt, MlpGradNorm("f16") as clip:
        clip.forward(g, norm)
        opt.step(g, 2.0 ** -7)
        torch.cuda.synchronize()
        assert abs(float(norm) - math.sqrt(sum((i + 1) ** 2 for i, k in enumerate(sizes) if k))) <= 2.0 ** -22 * float(norm)
        for t in w:
            assert t.numel() == 0 or abs(float(t) + 2.0 ** -7) <= 2.0 ** -7 * (2.0 ** -11 + 2.0 ** -20)
