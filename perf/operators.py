"""The operators around the two products of a transformer MLP block, as cases to time and check: layer norm and the
linear layer with bias, activation and residual, forward and backward.

`run` computes a case in plain torch (32 bits, rounded once at the end) or, where `own` is true, through this
package's `MlpNorm` and `MlpLinear`.  Widths are those of the package's workloads (512/2048, the 12288/6144,
8192/2752 and 8192/3584 shards)."""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5

# The ranges the listed cases stand for; a drawn case costs no more than the largest listed one of its operator.
MAX_ROWS = 8192
MAX_WIDTH = 12288
MAX_NORM = 8192 * 8192
MAX_FORWARD = 2048 * 6144 * 12288
MAX_BACKWARD = 2048 * 12288 * 6144


def listed():
    return [
        # one token through the smallest model's norm: a call is all latency
        {"name": "norm_fwd_1x512", "op": "norm_fwd", "dtype": "f16", "rows": 1, "H": 512},
        # an ordinary prefill or training batch at the widest hidden size
        {"name": "norm_fwd_2048x12288", "op": "norm_fwd", "dtype": "f16", "rows": 2048, "H": 12288},
        # the longest batch, bf16
        {"name": "norm_fwd_8192x8192", "op": "norm_fwd", "dtype": "bf16", "rows": 8192, "H": 8192},
        # a ragged training batch whose residual branch adds its gradient
        {"name": "norm_bwd_1000x8192", "op": "norm_bwd", "dtype": "bf16", "rows": 1000, "H": 8192, "dres": True},
        # an ordinary training batch at the widest hidden size
        {"name": "norm_bwd_2048x12288", "op": "norm_bwd", "dtype": "f16", "rows": 2048, "H": 12288, "dres": True},
        # decoding one token: the first product streams its weights
        {"name": "lin_fwd_1_gelu", "op": "lin_fwd", "dtype": "f16", "rows": 1, "K": 12288, "N": 6144,
         "act": "gelu_tanh", "bias": True, "residual": False, "save": False},
        # decoding a small batch: the second product adds bias and residual
        {"name": "lin_fwd_16_res", "op": "lin_fwd", "dtype": "bf16", "rows": 16, "K": 3584, "N": 8192,
         "act": "none", "bias": True, "residual": True, "save": False},
        # a ragged prefill through the gated product
        {"name": "lin_fwd_300_swiglu", "op": "lin_fwd", "dtype": "f16", "rows": 300, "K": 8192, "N": 2752,
         "act": "swiglu", "bias": False, "residual": False, "save": False},
        # a training batch's second product with bias and residual
        {"name": "lin_fwd_2048_res", "op": "lin_fwd", "dtype": "f16", "rows": 2048, "K": 6144, "N": 12288,
         "act": "none", "bias": True, "residual": True, "save": False},
        # a small model's training step: launches count
        {"name": "lin_bwd_64_gelu", "op": "lin_bwd", "dtype": "f16", "rows": 64, "K": 512, "N": 2048,
         "act": "gelu_tanh", "bias": True},
        # a ragged training batch through the gated product
        {"name": "lin_bwd_1000_swiglu", "op": "lin_bwd", "dtype": "bf16", "rows": 1000, "K": 8192, "N": 3584,
         "act": "swiglu", "bias": False},
        # a training batch at the widest sizes
        {"name": "lin_bwd_2048_gelu", "op": "lin_bwd", "dtype": "f16", "rows": 2048, "K": 12288, "N": 6144,
         "act": "gelu_tanh", "bias": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number of lo..hi, its logarithm uniform, rounded to a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v / step) * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "lin_fwd", "lin_bwd"])
    dtype = rng.choice(["f16", "bf16"])
    rows = _spread(rng, 1, MAX_ROWS)
    if op.startswith("norm"):
        H = _spread(rng, 64, MAX_WIDTH, rng.choice([1, 8, 64]))
        case = {"op": op, "dtype": dtype, "rows": min(rows, MAX_NORM // H), "H": H}
        return {**case, "dres": rng.random() < 0.5} if op == "norm_bwd" else case
    act = rng.choice(["none", "gelu_tanh", "swiglu"])
    g = 2 if act == "swiglu" else 1
    K, N = _spread(rng, 64, MAX_WIDTH, 8), _spread(rng, 64, MAX_WIDTH // g, 8)
    most = (MAX_FORWARD if op == "lin_fwd" else MAX_BACKWARD) // (K * N * g)
    case = {"op": op, "dtype": dtype, "rows": max(1, min(rows, most)), "K": K, "N": N, "act": act,
            "bias": rng.random() < 0.7}
    if op == "lin_fwd":
        case.update(residual=rng.random() < 0.5, save=rng.random() < 0.3)
    return case


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dt, dev = DTYPES[case["dtype"]], "cuda"
    gen = torch.Generator(dev).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    R = case["rows"]
    t = {}
    if case["op"].startswith("norm"):
        H = case["H"]
        # hidden states: channels with a mean and a spread of their own
        t["x"] = (normal(R, H) * (0.5 + normal(H).abs()) + 0.2 * normal(H)).to(dt)
        t["weight"] = (1 + 0.1 * normal(H)).to(dt)
        t["bias"] = (0.1 * normal(H)).to(dt)
        if case["op"] == "norm_bwd":
            t["dy"] = (0.1 * normal(R, H)).to(dt)
            t["dres"] = (0.1 * normal(R, H)).to(dt) if case["dres"] else None
            var, mean = torch.var_mean(t["x"].float(), 1, correction=0)
            t["mean"], t["rstd"] = mean, torch.rsqrt(var + EPS)
        return t
    K, N = case["K"], case["N"]
    gN = N * (2 if case["act"] == "swiglu" else 1)
    t["x"] = normal(R, K).to(dt)
    t["w"] = (normal(K, gN) / math.sqrt(K)).to(dt)
    t["bias"] = (0.1 * normal(gN)).to(dt) if case["bias"] else None
    if case["op"] == "lin_fwd":
        t["residual"] = normal(R, N).to(dt) if case["residual"] else None
    else:
        t["dy"] = (0.1 * normal(R, N)).to(dt)
        t["z"] = normal(R, gN).to(dt) if case["act"] != "none" else None
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    state = {"case": dict(case), "in": t}
    if not own:
        return state
    # what a user's program holds: the layer's handle and its output buffers
    from consumer_gemm_chain_amd import MlpLinear, MlpNorm
    R, op = case["rows"], case["op"]
    like = lambda *shape: torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")  # noqa: E731
    if op.startswith("norm"):
        state["layer"] = MlpNorm(case["H"], case["dtype"], EPS)
        if op == "norm_fwd":
            out = {"y": like(R, case["H"]), "mean": torch.empty(R, device="cuda"), "rstd": torch.empty(R, device="cuda")}
        else:
            out = {"dx": like(R, case["H"]), "dweight": like(case["H"]), "dbias": like(case["H"])}
    else:
        state["layer"] = MlpLinear(R, case["K"], case["N"], case["act"], case["dtype"])
        gN = t["w"].shape[1]
        if op == "lin_fwd":
            out = {"y": like(R, case["N"]), "z": like(R, gN) if case["save"] else None}
        else:
            out = {"dx": like(R, case["K"]), "dw": like(case["K"], gN), "db": like(gN) if case["bias"] else None}
    state["out"] = out
    return state


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    t, o, layer, op = state["in"], state["out"], state["layer"], state["case"]["op"]
    if op == "norm_fwd":
        layer.forward(t["x"], t["weight"], t["bias"], o["y"], o["mean"], o["rstd"])
    elif op == "norm_bwd":
        layer.backward(t["dy"], t["x"], t["weight"], t["mean"], t["rstd"], o["dx"], o["dweight"], o["dbias"],
                       dres=t["dres"])
    elif op == "lin_fwd":
        layer.forward(t["x"], t["w"], o["y"], bias=t["bias"], residual=t["residual"], z=o["z"])
    else:
        layer.backward(t["dy"], t["x"], t["w"], dx=o["dx"], dw=o["dw"], db=o["db"], z=t["z"])
    return o


def _gelu(h):
    return 0.5 * h * (1 + torch.tanh(math.sqrt(2 / math.pi) * (h + 0.044715 * h * h * h)))


def _run_plain(state):
    t, case = state["in"], state["case"]
    dt, op = DTYPES[case["dtype"]], case["op"]
    x = t["x"].float()
    if op == "norm_fwd":
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = torch.rsqrt((c * c).mean(1) + EPS)
        y = c * rstd[:, None] * t["weight"].float() + t["bias"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dy, rstd = t["dy"].float(), t["rstd"][:, None]
        xhat = (x - t["mean"][:, None]) * rstd
        g = dy * t["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if t["dres"] is not None:
            dx = dx + t["dres"].float()
        return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}
    N, act, w = case["N"], case["act"], t["w"].float()
    if op == "lin_fwd":
        h = x @ w
        if t["bias"] is not None:
            h = h + t["bias"].float()
        if act == "gelu_tanh":
            y = _gelu(h)
        elif act == "swiglu":
            y = h[:, :N] / (1 + torch.exp(-h[:, :N])) * h[:, N:]
        else:
            y = h
        if t["residual"] is not None:
            y = y + t["residual"].float()
        return {"y": y.to(dt), "z": h.to(dt) if case["save"] else None}
    dy = t["dy"].float()
    if act == "gelu_tanh":
        z = t["z"].float()
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        dz = dy * (0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z))
    elif act == "swiglu":
        gate, up = t["z"][:, :N].float(), t["z"][:, N:].float()
        s = 1 / (1 + torch.exp(-gate))
        dz = torch.cat([dy * up * s * (1 + gate * (1 - s)), dy * gate * s], 1)
    else:
        dz = dy
    return {"dx": (dz @ w.t()).to(dt), "dw": (x.t() @ dz).to(dt), "db": dz.sum(0).to(dt) if case["bias"] else None}


def exact(case, seed):
    """The outputs of `run` from the definitions in 64 bits, the gradients by differentiating the definitions."""
    t = {k: v.double() if v is not None else None for k, v in _inputs(case, seed).items()}
    op = case["op"]

    def norm(x, weight, bias):
        mean = x.sum(1, keepdim=True) / x.shape[1]
        sd = torch.sqrt(((x - mean) ** 2).sum(1, keepdim=True) / x.shape[1] + EPS)
        return (x - mean) / sd * weight + bias, mean[:, 0], 1 / sd[:, 0]

    def activation(z):
        if case["act"] == "gelu_tanh":
            u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            return z * torch.sigmoid(2 * u)
        if case["act"] == "swiglu":
            gate, up = z.split(case["N"], 1)
            return gate * torch.sigmoid(gate) * up
        return z

    if op == "norm_fwd":
        y, mean, rstd = norm(t["x"], t["weight"], t["bias"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        x, weight, bias = (t[k].requires_grad_() for k in ("x", "weight", "bias"))
        norm(x, weight, bias)[0].backward(t["dy"])
        dx = x.grad if t["dres"] is None else x.grad + t["dres"]
        return {"dx": dx, "dweight": weight.grad, "dbias": bias.grad}
    if op == "lin_fwd":
        z = torch.mm(t["x"], t["w"])
        if t["bias"] is not None:
            z += t["bias"]
        y = activation(z)
        if t["residual"] is not None:
            y = y + t["residual"]
        return {"y": y, "z": z if case["save"] else None}
    z = t["z"] if t["z"] is not None else torch.zeros_like(t["dy"])
    z.requires_grad_()
    dz, = torch.autograd.grad(activation(z), z, t["dy"]) if case["act"] != "none" else (t["dy"],)
    return {"dx": torch.mm(dz, t["w"].t()), "dw": torch.mm(t["x"].t(), dz),
            "db": dz.sum(0) if case["bias"] else None}


def work(case):
    R = case["rows"]
    if case["op"] == "norm_fwd":
        H = case["H"]
        return {"bytes": 2 * (2 * R * H + 2 * H) + 8 * R, "flops": 8 * R * H}
    if case["op"] == "norm_bwd":
        H = case["H"]
        return {"bytes": 2 * ((4 if case["dres"] else 3) * R * H + 3 * H) + 8 * R, "flops": 14 * R * H}
    K, N = case["K"], case["N"]
    gN = N * (2 if case["act"] == "swiglu" else 1)
    if case["op"] == "lin_fwd":
        values = R * K + K * gN + R * N
        values += (gN if case["bias"] else 0) + (R * N if case["residual"] else 0) + (R * gN if case["save"] else 0)
        return {"bytes": 2 * values, "flops": 2 * R * K * gN}
    values = R * N + 2 * R * K + 2 * K * gN + (R * gN if case["act"] != "none" else 0) + (gN if case["bias"] else 0)
    return {"bytes": 2 * values, "flops": 4 * R * K * gN}
