"""Gradient norm and AdamW on the GPU, through the binding, against the definitions.

Tolerances.  Norms are summed in 64 bits: one rounding to fp32.  AdamW's arithmetic is fp32: m and v are two products and
a sum (3 x 2^-24 of their terms), the weight's change a handful of operations with hardware root and reciprocal (2^-20 of
it), the weight one more rounding, and 16-bit weights one of theirs.  8-bit states are the fp32 ones rounded: m and v are
made again with the same fp32 operations, and codes have to be equal.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW, MlpGradNorm  # noqa: E402

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def gen(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g, device="cuda")


def off(t, shift):
    """`t` as a contiguous view `shift` elements into a buffer, and a check of what lies around it."""
    n = t.numel()
    base = torch.zeros(n + shift + 40, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device=t.device)
    base.view(torch.uint8).fill_(0x55)
    keep = base.clone()
    view = base[shift:shift + n].view(t.dtype)
    view.copy_(t.reshape(-1)) if t.element_size() > 1 else view.view(torch.uint8).copy_(t.reshape(-1).view(torch.uint8))

    def around():
        a, b = base.view(torch.uint8), keep.view(torch.uint8)
        lo, hi = shift * t.element_size(), (shift + n) * t.element_size()
        return torch.equal(a[:lo], b[:lo]) and torch.equal(a[hi:], b[hi:])
    return view.view(t.shape), around


# ------------------------------------------------------------------------ norm

def norm_of(grads, dtype, **kw):
    norm, scale = (torch.full((1,), 7.0, device="cuda") for _ in range(2))
    with MlpGradNorm(dtype) as layer:
        layer.forward(grads, norm, scale, **kw)
        torch.cuda.synchronize()
    return float(norm), float(scale)


def check_norm(sizes, dtype, shift=0, max_norm=1.0, unscale=1.0, size=1.0):
    n = gen(len(sizes))
    grads = [off((size * n(k)).to(DT[dtype]), shift + i % 3 if shift else 0)[0] for i, k in enumerate(sizes)]
    norm, scale = norm_of(grads, dtype, max_norm=max_norm, unscale=unscale)
    ref = abs(unscale) * math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(norm - ref) <= 2.0 ** -23 * ref
    ref_scale = unscale * min(1.0, max_norm / ref if ref else 1.0)
    assert abs(scale - ref_scale) <= 2.0 ** -23 * abs(ref_scale)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [7], [8], [512], [8191], [8192], [8193], [100003], [3, 1, 0, 5], [0, 0, 1],
                                   [512] * 183, [512] * 184, [512] * 185, [512] * 400, [5000, 1] * 200, [1 << 22, 3, 1 << 20]])
def test_grad_norm(sizes, dtype):
    check_norm(sizes, dtype)


@pytest.mark.parametrize("shift", [1, 3, 8])
def test_grad_norm_of_unaligned_tensors(shift):
    check_norm([5, 1000, 20011], "f16", shift)
    check_norm([5, 1000, 20011], "bf16", shift)


@pytest.mark.parametrize("max_norm,unscale", [(math.inf, 1.0), (1e-3, 1.0), (1e9, 1.0), (1.0, 2.0 ** -12), (5.0, -0.5)])
def test_grad_norm_scales(max_norm, unscale):
    check_norm([3000, 77], "f16", max_norm=max_norm, unscale=unscale)


def test_grad_norm_of_nothing():
    for grads in ([], [torch.empty(0, dtype=torch.float16, device="cuda")] * 3, [torch.zeros(999, dtype=torch.float16, device="cuda")]):
        assert norm_of(grads, "f16", max_norm=1.0, unscale=0.25) == (0.0, 0.25)


@pytest.mark.parametrize("size", [1e-25, 1e-20, 1e20, 1e30])
def test_grad_norm_far_from_one(size):
    """Squares outside fp32's range."""
    check_norm([5000, 3], "bf16", size=size, max_norm=size)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 4999, 5002])
def test_grad_norm_that_is_not_finite(bad, at):
    g = torch.ones(5003, dtype=torch.float16, device="cuda")
    g[at] = bad
    norm, scale = norm_of([g[:5000], g[5000:]], "f16", max_norm=1.0)
    assert not math.isfinite(norm) and math.isnan(scale)


def test_grad_norm_beyond_fp32():
    g = torch.full((100000,), 3e38, dtype=torch.bfloat16, device="cuda")
    norm, scale = norm_of([g], "bf16", max_norm=1.0)
    assert norm == math.inf and math.isnan(scale)


def test_grad_norm_twice_the_same():
    n = gen(3)
    grads = [n(k).half() for k in (100001, 3, 70000)]
    assert norm_of(grads, "f16") == norm_of(grads, "f16")


# ----------------------------------------------------------------------- adamw

def mix(x):
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def block_scale(x, exponent):
    """Of a vector: the power of two of each block of 256, from its finite values."""
    x = torch.nn.functional.pad(x.abs(), (0, -x.numel() % 256)).view(-1, 256)
    top = torch.where(torch.isfinite(x), x, 0.0).amax(1).double()
    e = torch.ceil(torch.log2(top / (1.75 * 2.0 ** exponent))).clamp(min=-126.0)
    return torch.where(top > 0, torch.exp2(e), 1.0).float()


def per_element(scale, n):
    return scale.repeat_interleave(256)[:n]


def v_codes(v, scale, t, seed, number):
    """e5m2 bytes of v in units of its block's scale: floor(y / step + u) steps."""
    n = v.numel()
    y = (v / per_element(scale, n)).double()
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -14))) - 2)
    place = torch.arange(n, device=v.device)
    key = mix(torch.tensor((int(mix(torch.tensor((t + seed) & 0xFFFFFFFF))) + 0x9E3779B9 * number) & 0xFFFFFFFF))
    r = mix(((place >> 1) + int(key)) & 0xFFFFFFFF)
    u = torch.where(place % 2 == 0, r & 0xFFFF, r >> 16).double() / 65536
    # (subnormal y is taken with 2^-14 added, in fp32)
    small = y < 2.0 ** -14
    y = torch.where(small, (y.float() + 2.0 ** -14).double() - 2.0 ** -14, y)
    q = torch.floor(y / step + u)
    q = torch.where((v > 0) & (q < 1), 1.0, q) * step
    q = torch.where(torch.isfinite(v), q, math.nan)
    return q.float()


class Case:
    """Tensors of an optimizer in the middle of a run, and what a step should make of them."""

    def __init__(self, sizes, dtype, bits, master, seed=1, shift=0, decay=0.1, b1=0.9, b2=0.95, eps=1e-8, size=1e-3):
        n = gen(seed)
        dt = DT[dtype]
        self.dtype, self.bits, self.b1, self.b2, self.eps, self.seed = dtype, bits, b1, b2, eps, 1000 + seed
        self.checks = []

        def place(t, i):
            v, ok = off(t, shift + i % 3 if shift else 0)
            self.checks.append(ok)
            return v
        spread = [size * (0.5 + n(k).abs()) for k in sizes]
        full = [n(k) for k in sizes]
        self.w = [place((0.02 * t).to(dt), i) for i, t in enumerate(full)]
        self.grad = [place((s * n(k)).to(dt), i) for i, (s, k) in enumerate(zip(spread, sizes))]
        self.master = [place(0.02 * t, i) for i, t in enumerate(full)] if master else None
        m = [0.3 * s * n(k) for s, k in zip(spread, sizes)]
        v = [(s * (0.5 + n(k).abs())) ** 2 for s, k in zip(spread, sizes)]
        self.m_scale = self.v_scale = None
        if bits == 8:
            self.m_scale = [place(block_scale(t, 8), i) for i, t in enumerate(m)]
            self.v_scale = [place(block_scale(t, 15), i) for i, t in enumerate(v)]
            m = [(t / per_element(s, t.numel())).to(E4) for t, s in zip(m, self.m_scale)]
            v = [(t / per_element(s, t.numel())).to(E5) for t, s in zip(v, self.v_scale)]
        self.m = [place(t, i) for i, t in enumerate(m)]
        self.v = [place(t, i) for i, t in enumerate(v)]
        self.decay = [decay * (i % 2) for i in range(len(sizes))]
        self.t = torch.tensor([41], device="cuda")

    def optimizer(self):
        return MlpAdamW(self.w, self.dtype, self.bits, self.b1, self.b2, self.eps, self.decay, self.seed, self.master, self.m,
                        self.v, self.m_scale, self.v_scale, self.t)

    def expected(self, lr, scale=1.0):
        """w before its rounding to 16 bits, its error, and m and v in fp32."""
        out = []
        t = int(self.t) + 1
        for i, g in enumerate(self.grad):
            k = g.numel()
            m, v = self.m[i].float(), self.v[i].float()
            if self.bits == 8:
                m, v = m * per_element(self.m_scale[i], k), v * per_element(self.v_scale[i], k)
            g = g.float() * scale
            m = m * self.b1 + g * (1 - self.b1)
            v = v * self.b2 + (g * g) * (1 - self.b2)
            w = (self.master[i] if self.master else self.w[i]).double()
            change = lr / (1 - self.b1 ** t) * m.double() / (torch.sqrt(v.double() / (1 - self.b2 ** t)) + self.eps)
            ref = w * (1 - lr * self.decay[i]) - change
            out.append((ref, 2.0 ** -20 * change.abs() + 2.0 ** -22 * w.abs() + 2.0 ** -23 * ref.abs(), m, v))
        return out

    def check(self, expected, number=0):
        u = U[self.dtype]
        for i, (ref, tol, m, v) in enumerate(expected):
            if self.master:
                assert ((self.master[i].double() - ref).abs() <= tol).all(), ("master", i)
                assert torch.equal(self.w[i], self.master[i].to(DT[self.dtype])), ("w", i)
            else:
                assert ((self.w[i].double() - ref).abs() <= tol + u * ref.abs() + 2.0 ** -25).all(), ("w", i)
            if self.bits == 32:
                assert torch.equal(self.m[i], m), ("m", i)
                assert torch.equal(self.v[i], v), ("v", i)
                continue
            ms, vs = block_scale(m, 8), block_scale(v, 15)
            assert torch.equal(self.m_scale[i], ms), ("m_scale", i)
            assert torch.equal(self.v_scale[i], vs), ("v_scale", i)
            k = m.numel()
            mm = torch.where(torch.isfinite(m), m / per_element(ms, k), math.nan).to(E4).float()
            assert torch.equal(self.m[i].float().nan_to_num(nan=1e9), mm.nan_to_num(nan=1e9)), ("m", i)
            vv = v_codes(v, vs, int(self.t), self.seed, number + i)
            assert torch.equal(self.v[i].float().nan_to_num(nan=1e9), vv.nan_to_num(nan=1e9)), ("v", i)
        assert all(ok() for ok in self.checks), "written around a tensor"


SIZES = [[1], [7], [8], [255], [256], [257], [2047], [2048], [2049], [100003], [3, 1, 0, 5, 700], [0], [600] * 47, [600] * 48,
         [600] * 49, [300, 9] * 60]


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_adamw(sizes, bits, master):
    for dtype in ("f16", "bf16"):
        c = Case(sizes, dtype, bits, master)
        expected = c.expected(1e-3)
        with c.optimizer() as opt:
            opt.step(c.grad, 1e-3)
            torch.cuda.synchronize()
        assert int(c.t) == 42
        c.check(expected)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 5, 8])
def test_adamw_of_unaligned_tensors(shift, bits):
    for master in (False, True):
        c = Case([5, 1000, 20011, 256], "bf16", bits, master, shift=shift)
        expected = c.expected(1e-3)
        with c.optimizer() as opt:
            opt.step(c.grad, 1e-3)
            torch.cuda.synchronize()
        c.check(expected)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_several_steps(bits):
    """Each from the states that the one before left; rates and scales of their own."""
    c = Case([3000, 40], "f16", bits, True)
    lr_scale = torch.ones(1, device="cuda")
    with c.optimizer() as opt:
        for k in range(4):
            scale = torch.tensor([0.5 + k], device="cuda")
            lr_scale.fill_(2.0 ** -k)
            expected = c.expected(1e-3 * 2.0 ** -k, 0.5 + k)
            opt.step(c.grad, 1e-3, scale=scale, lr_scale=lr_scale)
            torch.cuda.synchronize()
            c.check(expected)
    assert int(c.t) == 45


@pytest.mark.parametrize("kw", [{"b1": 0.0}, {"b2": 0.0}, {"b1": 0.0, "b2": 0.0}, {"b2": 0.9999}, {"eps": 1.0},
                                {"decay": 0.0}, {"size": 1e-18, "eps": 1e-30}, {"size": 1e15}])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_parameters(bits, kw):
    c = Case([1, 5000], "bf16", bits, True, **kw)
    expected = c.expected(1e-2)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-2)
        torch.cuda.synchronize()
    c.check(expected)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_first_step(bits):
    """States made by the optimizer: m = (1 - beta1) g, v = (1 - beta2) g^2, a change of lr in the gradient's direction."""
    n = gen(5)
    w, g = n(3000).half(), n(3000).half()
    before = w.clone()
    with MlpAdamW([w], "f16", bits, eps=0.0) as opt:
        opt.step([g], 0.25)
        torch.cuda.synchronize()
        assert int(opt.t) == 1
    ref = before.double() - 0.25 * torch.sign(g.double())
    assert ((w.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -19).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_leaves_a_step_out(bits, bad):
    c = Case([700, 3], "f16", bits, True)
    tensors = c.w + c.master + c.m + c.v + (c.m_scale + c.v_scale if bits == 8 else []) + [c.t]
    before = [t.clone() for t in tensors]
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3, scale=torch.tensor([bad], device="cuda"))
        torch.cuda.synchronize()
        for a, b in zip(tensors, before):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        expected = c.expected(1e-3)
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    c.check(expected)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_gradients_that_are_not_finite(bits, bad):
    """Their element is not finite any more; the others, those of its block too, are what they would be."""
    c = Case([700, 300], "bf16", bits, True)
    c.grad[0][300] = bad
    expected = c.expected(1e-3)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    assert not math.isfinite(float(c.w[0][300])) and not math.isfinite(float(c.master[0][300]))
    for t in (c.m[0], c.v[0]):
        assert not math.isfinite(float(t[300].float()))
    w, master = c.w[0].clone(), c.master[0].clone()
    ref, tol, m, v = expected[0]
    keep = torch.arange(700, device="cuda") != 300
    assert ((master.double() - ref).abs() <= tol)[keep].all() and torch.equal(w[keep], master[keep].to(w.dtype))
    if bits == 32:
        assert torch.equal(c.m[0][keep], m[keep]) and torch.equal(c.v[0][keep], v[keep])
    else:
        c.master[0].copy_(ref.float().nan_to_num())      # (the weights are looked at above)
        c.w[0].copy_(c.master[0].to(c.w[0].dtype))
        c.check([(c.master[0].double(), tol.nan_to_num(), m, v)] + expected[1:])


def test_adamw_zero_blocks_and_wide_ranges():
    """Blocks of zeros, and blocks whose numbers span more than 8 bits hold: none becomes zero in v, m rounds to zero."""
    c = Case([256 * 5], "bf16", 8, True)
    g = torch.zeros(256 * 5, device="cuda")
    g[256:512] = torch.logspace(-18, 18, 256, device="cuda")
    g[512:768] = torch.logspace(-37, -30, 256, device="cuda")
    g[768:1024] = 1.0
    c.grad[0].copy_(g)
    for t in (c.m[0], c.v[0]):
        t.view(torch.uint8)[:].zero_()
    for t in (c.m_scale[0], c.v_scale[0]):
        t.fill_(1.0)
    expected = c.expected(1e-3)
    with c.optimizer() as opt:
        opt.step(c.grad, 1e-3)
        torch.cuda.synchronize()
    v = c.v[0].float() * per_element(c.v_scale[0], 1280)
    assert (c.v[0].float()[expected[0][3] > 0] > 0).all() and (v[:256] == 0).all() and (v[1024:] == 0).all()
    assert float(c.m_scale[0][0]) == 1.0 and float(c.v_scale[0][4]) == 1.0
    c.check(expected)


def test_adamw_rounds_v_by_chance_without_bias():
    """Over many elements the rounding of v has a mean of zero, and it differs from step to step."""
    n = 1 << 20
    n_ = gen(9)
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    v0 = 2.0 ** -20 * (1 + 0.7 * torch.rand(n, generator=torch.Generator("cuda").manual_seed(1), device="cuda"))
    moved = []
    w = (0.02 * n_(n)).bfloat16()
    for seed in (1, 2):
        code = (v0 / 2.0 ** -35).to(E5)
        scale = torch.full((n // 256,), 2.0 ** -35, device="cuda")
        before = code.float().double()
        with MlpAdamW([w.clone()], "bf16", 8, beta2=0.99, seed=seed, v=[code], v_scale=[scale]) as opt:
            opt.step([grad], 0.0)
            torch.cuda.synchronize()
        after = opt.v[0].float().double() * per_element(opt.v_scale[0], n).double() / 2.0 ** -35
        moved.append(after != before)
        # a step of e5m2 is at most 0.25 of the number: so is each error, and their mean below six sigma
        error = after / (0.99 * before) - 1
        assert float(error.abs().max()) <= 0.26
        assert abs(float(error.mean())) <= 6 * 0.25 / math.sqrt(n)
    assert 0 < float(moved[0].double().mean()) < 1 and bool((moved[0] != moved[1]).any())


# ------------------------------------------------------------- graphs and refusals

def states_of(c):
    return c.w + (c.master or []) + c.m + c.v + (c.m_scale or []) + (c.v_scale or []) + [c.t]


@pytest.mark.parametrize("bits", [32, 8])
def test_step_graph_replays(bits):
    """Norm and step captured once; each replay takes the next step, as eager calls do, a schedule and a step that is left
    out among them."""
    sizes = [3000, 40] * 30
    a, b = (Case(sizes, "f16", bits, True, seed=3) for _ in range(2))
    norm, scale, lr_scale = (torch.ones(1, device="cuda") for _ in range(3))
    with a.optimizer() as eager, b.optimizer() as graphed, MlpGradNorm("f16") as clip:
        keep = [t.clone() for t in states_of(b)]

        def step(c, opt):
            clip.forward(c.grad, norm, scale, max_norm=0.1)
            opt.step(c.grad, 1e-2, scale=scale, lr_scale=lr_scale)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step(b, graphed)
        torch.cuda.synchronize()
        for t, k in zip(states_of(b), keep):
            t.copy_(k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(b, graphed)
        n = gen(4)
        for k in range(4):
            lr_scale.fill_(0.5 ** k)
            for x, y in zip(a.grad, b.grad):
                x.copy_(1e-3 * n(x.numel()))
                if k == 2:
                    x[0] = math.inf
                y.copy_(x)
            step(a, eager)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(states_of(a), states_of(b)):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), k
    assert int(b.t) == 44


def test_optimizers_on_two_streams_at_once():
    cases = [Case([5000, 300], "bf16", 8, True, seed=k) for k in (1, 2)]
    expected = [c.expected(1e-3) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    opts = [c.optimizer() for c in cases]
    torch.cuda.synchronize()
    for c, s, opt in zip(cases, streams, opts):
        with torch.cuda.stream(s):
            opt.step(c.grad, 1e-3)
    torch.cuda.synchronize()
    for c, e, opt in zip(cases, expected, opts):
        c.check(e)
        opt.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_on_another_stream_than_the_optimizer_was_made_on(bits):
    """States and master weights are there when the constructor returns."""
    n = gen(3)
    w = [(0.02 * n(k)).half() for k in (1 << 20, 300)]
    g = [(1e-3 * n(k)).half() for k in (1 << 20, 300)]

    def step(make, run):
        params = [t.clone() for t in w]
        slow = n(4096, 4096)
        torch.cuda.synchronize()
        with torch.cuda.stream(make):
            for _ in range(10):
                slow = slow @ slow
            opt = MlpAdamW(params, "f16", bits, master=True)
        with torch.cuda.stream(run):
            opt.step(g, 1e-3)
        torch.cuda.synchronize()
        state = opt.params + opt.master + opt.m + opt.v + (opt.m_scale or []) + (opt.v_scale or []) + [opt.t]
        opt.close()
        return [t.view(torch.uint8) for t in state]
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    for a, b in zip(step(here, there), step(here, here)):
        assert torch.equal(a, b)


def test_parameters_that_require_gradients():
    """Master weights are plain tensors, not part of a graph."""
    w = torch.nn.Parameter(torch.randn(300, device="cuda").half())
    with MlpAdamW([w], "f16", master=True) as opt:
        assert not opt.master[0].requires_grad
        opt.step([torch.ones_like(w)], 1e-2)
        torch.cuda.synchronize()
        assert torch.equal(opt.master[0].half(), w.detach())


def test_tensors_of_any_shape():
    n = gen(6)
    w = n(30, 17).half()
    g = n(30, 17).half()
    flat, gflat = w.clone().view(-1), g.view(-1)
    with MlpAdamW([w], "f16", 8) as a, MlpAdamW([flat], "f16", 8) as b:
        a.step([g], 1e-2)
        b.step([gflat], 1e-2)
        torch.cuda.synchronize()
        assert a.m[0].shape == w.shape
    assert torch.equal(w.view(-1), flat)


def test_refusals_of_tensors():
    w = [torch.randn(64, 8, device="cuda").half(), torch.randn(9, device="cuda").half()]
    g = [torch.randn_like(t) for t in w]
    for bad, needle in (({"states": 16}, "32 or 8"), ({"beta1": 1.0}, "beta"), ({"eps": -1.0}, "eps"), ({"decay": [0.1]}, "decay has"),
                        ({"master": [w[0].float()]}, "master must have"), ({"m": [t.float()[:3] for t in w]}, "m must have"),
                        ({"m": w}, "float32"), ({"step": torch.zeros(1, dtype=torch.int32, device="cuda")}, "int64"),
                        ({"states": 8, "m_scale": [torch.ones(3, device="cuda")] * 2}, "m_scale must have")):
        with pytest.raises((ValueError, Exception), match=needle):
            MlpAdamW(w, "f16", **bad)
    with pytest.raises(ValueError, match="twice"):
        MlpAdamW([w[0], w[1], w[0]], "f16")
    with pytest.raises(ValueError, match="contiguous"):
        MlpAdamW([w[0].t()], "f16")
    with pytest.raises(ValueError, match="device"):
        MlpAdamW([w[0].cpu()], "f16")
    one = torch.ones(1, device="cuda")
    with MlpAdamW(w, "f16") as opt, MlpGradNorm("f16") as clip:
        for grads, needle in (([g[0]], "shapes"), ([g[1], g[0]], "shapes"), ([g[0].t().contiguous(), g[1]], "shapes"),
                              ([g[0].float(), g[1]], "float16"), ([g[0].cpu(), g[1]], "device"),
                              ([torch.randn(8, 64, device="cuda").half().t(), g[1]], "contiguous")):
            with pytest.raises(ValueError, match=needle):
                opt.step(grads, 1e-3)
        with pytest.raises(ValueError, match="scale"):
            opt.step(g, 1e-3, scale=one.cpu())
        with pytest.raises(ValueError, match="scale"):
            opt.step(g, 1e-3, scale=torch.ones((), device="cuda"))
        with pytest.raises(Exception, match="lr"):
            opt.step(g, math.inf)
        with pytest.raises(ValueError, match="float16"):
            clip.forward([g[0].float()], one)
        with pytest.raises(ValueError, match="contiguous"):
            clip.forward([g[0].t()], one)
        with pytest.raises(Exception, match="max_norm"):
            clip.forward(g, one, max_norm=0.0)
        with pytest.raises(Exception, match="unscale"):
            clip.forward(g, one, unscale=0.0)
        opt.step(g, 1e-3)
        w[1].data = torch.zeros_like(w[1])
        with pytest.raises(ValueError, match="other memory"):
            opt.step(g, 1e-3)
        torch.cuda.synchronize()
