"""The operators that turn the MLP block's training pass into a training step, as cases to time and check: the softmax
cross entropy of a vocabulary head without its logits, with its gradient, the norm of all gradients, and an AdamW step
over many tensors with states in 32 or 8 bits.

`run` computes a case in plain torch or, where `own` is true, through this package's `MlpLoss`, `MlpGradNorm` and
`MlpAdamW`.  Hidden and inner widths are those of the package's workloads (512/2048, the 12288/6144 and 8192/3584 shards); vocabularies are
generic, odd ones among them."""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
B1, B2, EPS, LR, MAX_NORM = 0.9, 0.95, 1e-8, 1e-4, 1.0
BLOCK = 256        # elements that share a scale in 8-bit states
SEED = 12345       # of the 8-bit states' rounding

# The ranges the listed cases stand for; a drawn case costs no more than the largest listed one of its operator.
MAX_ROWS, MAX_VOCABULARY, MAX_WIDTH = 4096, 128000, 12288
MAX_HEAD = 8192 * 128000
MAX_PRODUCT = 4096 * 8192 * 128000
MAX_PARAMS = 150_000_000


def listed():
    return [
        # scoring one token with the smallest model: a call is all latency
        {"name": "loss_fwd_1x512", "op": "loss_fwd", "dtype": "f16", "rows": 1, "H": 512, "V": 1000, "ignored": 0.0},
        # scoring a small batch of tokens: the head's weights stream through
        {"name": "loss_fwd_48x8192", "op": "loss_fwd", "dtype": "bf16", "rows": 48, "H": 8192, "V": 32000,
         "ignored": 0.0},
        # evaluation or the forward half of a training step: a batch over a large vocabulary
        {"name": "loss_fwd_4096x8192", "op": "loss_fwd", "dtype": "bf16", "rows": 4096, "H": 8192, "V": 128000,
         "ignored": 0.1},
        # a small model's training step: launches count
        {"name": "loss_bwd_64x512", "op": "loss_bwd", "dtype": "f16", "rows": 64, "H": 512, "V": 1000, "ignored": 0.0,
         "zloss": False},
        # a ragged batch at the widest hidden size over an odd vocabulary, a third of its tokens left out (a prompt)
        {"name": "loss_bwd_1000x12288", "op": "loss_bwd", "dtype": "f16", "rows": 1000, "H": 12288, "V": 50001,
         "ignored": 0.33, "zloss": False},
        # a training batch over a large vocabulary, with a loss on the normaliser too
        {"name": "loss_bwd_4096x8192", "op": "loss_bwd", "dtype": "bf16", "rows": 4096, "H": 8192, "V": 128000,
         "ignored": 0.1, "zloss": True},
        # one small block's parameters, no fp32 copy of the weights
        {"name": "adamw32_512x1", "op": "adamw", "dtype": "f16", "H": 512, "I": 2048, "layers": 1, "bits": 32,
         "master": False},
        # one shard's block at the widest hidden size, fp32 master weights
        {"name": "adamw32_12288x1", "op": "adamw", "dtype": "bf16", "H": 12288, "I": 6144, "layers": 1, "bits": 32,
         "master": True},
        # a small model's many tensors, states in 8 bits
        {"name": "adamw8_512x24", "op": "adamw", "dtype": "bf16", "H": 512, "I": 2048, "layers": 24, "bits": 8,
         "master": False},
        # a shard of two layers, states in 8 bits beside fp32 master weights
        {"name": "adamw8_8192x2", "op": "adamw", "dtype": "bf16", "H": 8192, "I": 3584, "layers": 2, "bits": 8,
         "master": True},
        # the gradient norm of a small model's many tensors
        {"name": "grad_norm_512x24", "op": "grad_norm", "dtype": "f16", "H": 512, "I": 2048, "layers": 24},
        # the gradient norm of one shard's block
        {"name": "grad_norm_12288x1", "op": "grad_norm", "dtype": "bf16", "H": 12288, "I": 6144, "layers": 1},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number of lo..hi, its logarithm uniform, rounded to a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["loss_fwd", "loss_bwd", "adamw", "adamw", "grad_norm"])
    dtype = rng.choice(["f16", "bf16"])
    if op.startswith("loss"):
        H = _spread(rng, 64, MAX_WIDTH, 8)
        V = min(_spread(rng, 100, MAX_VOCABULARY), MAX_HEAD // H)
        rows = min(_spread(rng, 1, MAX_ROWS), MAX_PRODUCT // (H * V))
        case = {"op": op, "dtype": dtype, "rows": rows, "H": H, "V": V, "ignored": rng.choice([0.0, 0.1, 0.5])}
        return {**case, "zloss": rng.random() < 0.5} if op == "loss_bwd" else case
    H, I = _spread(rng, 64, MAX_WIDTH, rng.choice([1, 8, 64])), _spread(rng, 64, MAX_WIDTH, rng.choice([1, 8, 64]))
    most = max(1, min(32, MAX_PARAMS // (2 * H * I)))
    case = {"op": op, "dtype": dtype, "H": min(H, MAX_PARAMS // (2 * I)), "I": I, "layers": _spread(rng, 1, most)}
    return {**case, "bits": rng.choice([32, 8]), "master": rng.random() < 0.5} if op == "adamw" else case


# ------------------------------------------------------------------------ inputs

def _generator(seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return gen, lambda *shape: torch.randn(shape, generator=gen, device="cuda")


def _loss_inputs(case, seed):
    gen, normal = _generator(seed)
    dt, R, H, V = DTYPES[case["dtype"]], case["rows"], case["H"], case["V"]
    # logits of a spread of 3, the target's among the largest: hidden states lean towards their target's row
    w = (normal(V, H) * (3 / math.sqrt(H))).to(dt)
    target = torch.randint(V, (R,), generator=gen, device="cuda")
    x = (normal(R, H) + 5 * torch.rand((R, 1), generator=gen, device="cuda") * w[target].float() / 3).to(dt)
    target = torch.where(torch.rand(R, generator=gen, device="cuda") < case["ignored"], -1, target)
    t = {"x": x, "w": w, "target": target}
    if case["op"] == "loss_bwd":
        counted = (target >= 0).float()
        # the mean over the rows that count, in fp16 times a loss scale
        t["dloss"] = counted / counted.sum().clamp(min=1) * (4096 if case["dtype"] == "f16" else 1)
        z = x.float() @ w.float().t()
        top = z.max(1, keepdim=True)[0]
        t["lse"] = z.sub_(top).exp_().sum(1).log() + top[:, 0]
        # of 1e-4 times the normaliser's square
        t["dlse"] = 2e-4 * t["lse"] * t["dloss"] if case["zloss"] else None
    return t


def _shapes(case):
    """The tensors of the block's layers: norm scale and shift, two weights with their biases."""
    H, I = case["H"], case["I"]
    return [(H,), (H,), (H, I), (I,), (I, H), (H,)] * case["layers"]


def _decays(case):
    """Weight decay of each: of the two matrices only."""
    return [0.1 if len(s) == 2 else 0.0 for s in _shapes(case)]


def _starts(case):
    """Where each tensor begins in buffers that hold all of them, at whole blocks, and their length."""
    at, starts = 0, []
    for s in _shapes(case):
        starts.append(at)
        at += -(-math.prod(s) // BLOCK) * BLOCK
    return starts, at


def _views(case, flat):
    return [flat[a:a + math.prod(s)].view(s) for a, s in zip(_starts(case)[0], _shapes(case))]


def _e4m3_scale(top):
    """The power of two that brings a block's largest magnitude into the upper binade of e4m3 (largest 448); 1 for zeros."""
    return _scale(top, 8)


def _e5m2_scale(top):
    """The same for e5m2 (largest 57344)."""
    return _scale(top, 15)


def _scale(top, exponent):
    m, e = torch.frexp(top)                     # top = m 2^e, m in [1/2, 1)
    e = (e - 1 - exponent + (m > 0.875).to(e.dtype)).clamp(min=-126)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e.to(top.dtype)), 1.0)


def _params_inputs(case, seed):
    """Flat buffers: gradients, weights, and states as after a number of steps."""
    gen, normal = _generator(seed)
    dt, n = DTYPES[case["dtype"]], _starts(case)[1]
    there = torch.zeros(n, dtype=torch.bool, device="cuda")     # false between the tensors
    spread = torch.zeros(n, device="cuda")
    for v, s in zip(_views(case, there), _views(case, spread)):
        v.fill_(True)
        # each tensor's gradients have a size of their own, and so has each row
        s.copy_(10.0 ** (-3 + float(torch.randn((), generator=gen, device="cuda")) / 2) * (0.5 + normal(s.shape[0]).abs()).view(-1, *[1] * (s.dim() - 1)))
    grad = (normal(n) * spread).to(dt)
    t = {"grad": grad}
    if case["op"] == "grad_norm":
        return t
    master = normal(n) * 0.02 * there
    t["w"] = master.to(dt)
    t["master"] = master if case["master"] else None
    m = normal(n) * spread * 0.3
    v = (spread * (0.5 + torch.rand(n, generator=gen, device="cuda"))) ** 2
    t["step"] = torch.tensor([100 + seed % 100], device="cuda")
    t["scale"] = torch.rand((1,), generator=gen, device="cuda") + 0.5       # of the gradients: as a clipped norm gives it
    if case["bits"] == 32:
        return {**t, "m": m, "v": v}
    for name, x, scale, kind in (("m", m, _e4m3_scale, torch.float8_e4m3fn), ("v", v, _e5m2_scale, torch.float8_e5m2)):
        x = x.view(-1, BLOCK)
        t[name + "_scale"] = scale(x.abs().amax(1))
        t[name] = (x / t[name + "_scale"][:, None]).to(kind).view(-1)
    return t


def prepare(case, seed):
    loss = case["op"].startswith("loss")
    t = _loss_inputs(case, seed) if loss else _params_inputs(case, seed)
    state = {"case": dict(case), "in": t}
    if not own:
        if case["op"] == "adamw":
            # of each block: its tensor's number, decay, and the place of its first element in it
            starts, n = _starts(case)
            at = torch.arange(0, n, BLOCK, device="cuda")
            begin = torch.tensor(starts, device="cuda")
            which = torch.bucketize(at, begin, right=True) - 1
            state["blocks"] = {"which": which, "first": at - begin[which],
                               "decay": torch.tensor(_decays(case), dtype=torch.float64, device="cuda")[which]}
        return state
    # what a user's program holds: the handle and its output buffers, or the optimizer with its states
    from consumer_gemm_chain_amd import MlpAdamW, MlpGradNorm, MlpLoss
    dt = DTYPES[case["dtype"]]
    if loss:
        R, H, V = case["rows"], case["H"], case["V"]
        state["layer"] = MlpLoss(R, H, V, case["dtype"], grad=case["op"] == "loss_bwd")
        if case["op"] == "loss_fwd":
            state["out"] = {"loss": torch.empty(R, device="cuda"), "lse": torch.empty(R, device="cuda")}
        else:
            state["out"] = {"dx": torch.empty(R, H, dtype=dt, device="cuda"), "dw": torch.empty(V, H, dtype=dt, device="cuda")}
        return state
    state["grads"] = _views(case, t["grad"])
    if case["op"] == "grad_norm":
        state["layer"] = MlpGradNorm(case["dtype"])
        state["out"] = {"norm": torch.empty(1, device="cuda"), "scale": torch.empty(1, device="cuda")}
        return state
    each = {k: _views(case, t[k]) for k in ("w", "m", "v")}
    scales = None
    if case["bits"] == 8:
        counts = [-(-math.prod(s) // BLOCK) for s in _shapes(case)]
        scales = [[t[k][a // BLOCK:a // BLOCK + c] for a, c in zip(_starts(case)[0], counts)] for k in ("m_scale", "v_scale")]
    state["opt"] = MlpAdamW(each["w"], case["dtype"], states=case["bits"], beta1=B1, beta2=B2, eps=EPS, decay=_decays(case),
                            seed=SEED, master=_views(case, t["master"]) if case["master"] else None,
                            m=each["m"], v=each["v"], m_scale=scales and scales[0], v_scale=scales and scales[1], step=t["step"])
    return state


# ------------------------------------------------------------------------ passes

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _state_of(t):
    """What a step changes."""
    return {k: t[k] for k in ("w", "master", "m", "v", "m_scale", "v_scale", "step") if t.get(k) is not None}


def _run_own(state):
    t, op = state["in"], state["case"]["op"]
    if op == "loss_fwd":
        state["layer"].forward(t["x"], t["w"], t["target"], state["out"]["loss"], state["out"]["lse"])
    elif op == "loss_bwd":
        state["layer"].backward(t["x"], t["w"], t["target"], t["lse"], t["dloss"], t["dlse"], dx=state["out"]["dx"],
                                dw=state["out"]["dw"])
    elif op == "grad_norm":
        state["layer"].forward(state["grads"], state["out"]["norm"], state["out"]["scale"], max_norm=MAX_NORM)
    else:
        state["opt"].step(state["grads"], LR, scale=t["scale"])
        return _state_of(t)
    return state["out"]


def _run_plain(state):
    op, t = state["case"]["op"], state["in"]
    if op == "adamw":
        return _plain_adamw(state)
    if op == "grad_norm":
        norm = t["grad"].double().square().sum().sqrt()
        # not finite: the scale says so, and a step with it is left out
        scale = torch.where(norm < math.inf, (MAX_NORM / norm).clamp(max=1.0), math.nan)
        return {"norm": norm.float().view(1), "scale": scale.float().view(1)}
    x, w, target = t["x"].float(), t["w"].float(), t["target"]
    z = x @ w.t()
    at = target.clamp(min=0)[:, None]
    if op == "loss_fwd":
        z_at = z.gather(1, at)[:, 0]
        top = z.max(1, keepdim=True)[0]
        lse = (z - top).exp().sum(1).log() + top[:, 0]
        # rows that are left out: zeros
        return {"loss": torch.where(target >= 0, lse - z_at, 0.0), "lse": torch.where(target >= 0, lse, 0.0)}
    dloss, dt = torch.where(target >= 0, t["dloss"], 0.0), t["x"].dtype
    p = torch.exp(z - t["lse"][:, None])
    dlse = torch.where(target >= 0, t["dlse"], 0.0) if t["dlse"] is not None else torch.zeros_like(dloss)
    dz = p * (dloss + dlse)[:, None]
    dz.scatter_add_(1, at, -dloss[:, None])
    return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt)}


def _mix(x):
    """32 well mixed bits of 32 (in 64-bit integers, whose products wrap)."""
    x = ((x ^ (x >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random16(step, which, first):
    """The 16 random bits of each element of the blocks: of its pair's 32, the lower half's for the even place."""
    key = _mix((_mix((step + SEED) & 0xFFFFFFFF) + 0x9E3779B9 * which) & 0xFFFFFFFF)
    pair = (first[:, None] + torch.arange(0, BLOCK, 2, device=first.device)) >> 1
    r = _mix((pair + key[:, None]) & 0xFFFFFFFF)
    return torch.stack([r & 0xFFFF, r >> 16], 2).view(-1, BLOCK)


def _plain_adamw(state):
    case, t, blocks = state["case"], state["in"], state["blocks"]
    dt = DTYPES[case["dtype"]]
    t["step"] += 1
    step = t["step"].double()
    size = (LR / (1 - B1 ** step)).float()
    root = torch.sqrt(1 - B2 ** step).float()
    keep = (1 - LR * blocks["decay"]).float()[:, None]
    g = (t["grad"].float() * t["scale"]).view(-1, BLOCK)
    w = (t["master"] if case["master"] else t["w"].float()).view(-1, BLOCK)
    m, v = t["m"].float().view(-1, BLOCK), t["v"].float().view(-1, BLOCK)
    if case["bits"] == 8:
        m, v = m * t["m_scale"][:, None], v * t["v_scale"][:, None]
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    w = w * keep - size * (m / (torch.sqrt(v) / root + EPS))
    if case["master"]:
        t["master"].copy_(w.view(-1))
    t["w"].copy_(w.to(dt).view(-1))
    if case["bits"] == 32:
        t["m"].copy_(m.view(-1))
        t["v"].copy_(v.view(-1))
        return _state_of(t)
    t["m_scale"].copy_(_e4m3_scale(m.abs().amax(1)))
    t["m"].copy_((m / t["m_scale"][:, None]).to(torch.float8_e4m3fn).view(-1))
    # v: rounded up or down by chance, so that its mean moves though one step changes it by less than a rounding;
    # what is not zero stays at least the smallest number
    t["v_scale"].copy_(_e5m2_scale(v.amax(1)))
    y = v / t["v_scale"][:, None]
    small = y < 2.0 ** -14
    bits = (y + torch.where(small, 2.0 ** -14, 0.0)).view(torch.int32)
    r = _random16(t["step"], blocks["which"], blocks["first"]).to(torch.int32)
    code = ((bits + (r << 5)) >> 21) - (112 << 2) - torch.where(small, 4, 0)
    code = torch.where(y > 0, code.clamp(min=1), 0)
    t["v"].copy_(code.to(torch.uint8).view(torch.float8_e5m2).view(-1))
    return _state_of(t)


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    """The outputs of `run` from the definitions in 64 bits, the loss's gradients row by row of the definition."""
    if case["op"].startswith("loss"):
        return _exact_loss(case, seed)
    t = _params_inputs(case, seed)
    if case["op"] == "grad_norm":
        norm = torch.linalg.vector_norm(t["grad"].double())
        return {"norm": norm.view(1), "scale": torch.minimum(torch.ones_like(norm), MAX_NORM / norm).view(1)}
    n = int(t["step"]) + 1
    blocks = [-(-math.prod(s) // BLOCK) for s in _shapes(case)]
    count = torch.tensor(blocks, device="cuda")
    per_element = lambda v: torch.repeat_interleave(v, count * BLOCK)  # noqa: E731
    spread = lambda v: torch.repeat_interleave(v.double(), BLOCK)  # noqa: E731
    g = t["grad"].double() * t["scale"].double()
    m, v = t["m"].double(), t["v"].double()
    if case["bits"] == 8:
        m, v = m * spread(t["m_scale"]), v * spread(t["v_scale"])
    m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g ** 2
    w = t["master"].double() if case["master"] else t["w"].double()
    decay = per_element(torch.tensor(_decays(case), dtype=torch.float64, device="cuda"))
    w = w - LR * decay * w - LR * (m / (1 - B1 ** n)) / (torch.sqrt(v / (1 - B2 ** n)) + EPS)
    out = {"w": w, "step": torch.tensor([n], device="cuda")}
    if case["master"]:
        out["master"] = w
    if case["bits"] == 32:
        return {**out, "m": m, "v": v}

    def held(x, largest, fraction, lowest, u):
        """x in units of its block's scale, rounded to `fraction` bits: to the nearest, or with u down to below it."""
        top = x.abs().view(-1, BLOCK).amax(1)
        scale = torch.exp2(torch.ceil(torch.log2(top / largest)))
        scale = torch.where(top > 0, scale, 1.0)
        y = x / spread(scale)
        at = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** lowest))) - fraction)
        q = torch.round(y / at) if u is None else torch.floor(y / at + u)
        return scale, torch.where(y == 0, 0.0, q if u is None else q.clamp(min=1)) * at

    # (a block's elements may not lie in pairs across two tensors: places count from the tensor's start)
    starts = torch.cumsum(count * BLOCK, 0) - count * BLOCK
    place = torch.arange(g.numel(), device="cuda") - per_element(starts)

    def mixed(x):
        for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85)):
            x = torch.bitwise_xor(x, x >> shift) * factor % 2 ** 32
        return torch.bitwise_xor(x, x >> 16)

    key = mixed((mixed(torch.tensor(n + SEED, device="cuda")) + 0x9E3779B9 * torch.arange(len(blocks), device="cuda")) % 2 ** 32)
    bits = mixed((place // 2 + per_element(key)) % 2 ** 32)
    u = torch.where(place % 2 == 0, bits % 2 ** 16, bits // 2 ** 16).double() / 2 ** 16
    out["m_scale"], out["m"] = held(m, 448.0, 3, -6, None)
    out["v_scale"], out["v"] = held(v, 57344.0, 2, -14, u)
    return out


def _exact_loss(case, seed):
    t = _loss_inputs(case, seed)
    x, w, target = t["x"].double(), t["w"].double(), t["target"]
    z = torch.mm(x, w.t())
    counted = target >= 0
    if case["op"] == "loss_fwd":
        lse = torch.logsumexp(z, 1)
        picked = z[torch.arange(len(target), device=z.device), target.clamp(min=0)]
        return {"loss": (lse - picked) * counted, "lse": lse * counted}
    # p from the lse that the gradient is given
    z = torch.exp_(z.sub_(t["lse"].double()[:, None]))
    a = t["dloss"].double() + (t["dlse"].double() if t["dlse"] is not None else 0.0)
    z.mul_((a * counted)[:, None])
    rows = torch.nonzero(counted)[:, 0]
    z[rows, target[rows]] -= t["dloss"].double()[rows]
    return {"dx": torch.mm(z, w), "dw": torch.mm(z.t(), x)}


def work(case):
    if case["op"].startswith("loss"):
        R, H, V = case["rows"], case["H"], case["V"]
        counted = max(1, round(R * (1 - case["ignored"])))      # rows that are left out need no products
        if case["op"] == "loss_fwd":
            return {"bytes": 2 * H * (counted + V) + 16 * R, "flops": 2 * counted * H * V}
        return {"bytes": 2 * H * (counted + V) + 2 * H * (R + V) + (20 if case["zloss"] else 16) * R,
                "flops": 6 * counted * H * V}
    n = sum(math.prod(s) for s in _shapes(case))
    if case["op"] == "grad_norm":
        return {"bytes": 2 * n, "flops": 2 * n}
    weights = 10 if case["master"] else 4
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 + weights + states), "flops": 15 * n}
