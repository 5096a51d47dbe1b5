"""Whole training steps: the pre-norm MLP block, a norm, the vocabulary's cross entropy, the gradient norm and AdamW
together, against 64-bit autograd of the same model and AdamW by its formula."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW, MlpBlock, MlpGradNorm, MlpLoss, MlpNorm  # noqa: E402

ROWS, H, I, V, EPS = 200, 256, 512, 1003, 1e-5


class Model:
    """y = block(x); loss = cross entropy of norm(y) with a head W [V, H], mean over the rows that count."""

    def __init__(self, dtype, act, bits):
        dt = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        g = torch.Generator("cuda").manual_seed(1)
        n = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
        gI = 2 * I if act == "swiglu" else I
        self.dtype, self.act = dtype, act
        self.block_params = {"weight": 1 + 0.1 * n(H), "bias": 0.1 * n(H), "w1": n(H, gI) * H ** -0.5, "b1": 0.1 * n(gI),
                             "w2": n(I, H) * I ** -0.5, "b2": 0.1 * n(H)}
        self.block_params = {k: v.to(dt) for k, v in self.block_params.items()}
        self.head = {"weight": (1 + 0.1 * n(H)).to(dt), "bias": (0.1 * n(H)).to(dt), "w": (n(V, H) * H ** -0.5).to(dt)}
        self.params = list(self.block_params.values()) + list(self.head.values())
        self.block, self.norm = MlpBlock(ROWS, H, I, act, dtype, EPS), MlpNorm(H, dtype, EPS)
        self.loss, self.clip = MlpLoss(ROWS, H, V, dtype), MlpGradNorm(dtype)
        decay = [0.1 if p.dim() == 2 else 0.0 for p in self.params]
        self.opt = MlpAdamW(self.params, dtype, bits, 0.9, 0.95, 1e-8, decay, seed=7, master=True)
        self.scale_of_loss = 1024.0 if dtype == "f16" else 1.0

    def gradients(self, x, target):
        y, saved = self.block.forward(x, self.block_params, save=True)
        h, mean, rstd = torch.empty_like(y), *(torch.empty(ROWS, device="cuda") for _ in range(2))
        self.norm.forward(y, self.head["weight"], self.head["bias"], h, mean, rstd)
        loss, lse = (torch.empty(ROWS, device="cuda") for _ in range(2))
        self.loss.forward(h, self.head["w"], target, loss, lse)
        counted = (target >= 0).float()
        dloss = counted * (self.scale_of_loss / counted.sum())
        dh, dw, dy = torch.empty_like(h), torch.empty_like(self.head["w"]), torch.empty_like(y)
        dweight, dbias = torch.empty_like(self.head["weight"]), torch.empty_like(self.head["bias"])
        self.loss.backward(h, self.head["w"], target, lse, dloss, dx=dh, dw=dw)
        self.norm.backward(dh, y, self.head["weight"], mean, rstd, dy, dweight, dbias)
        _, grads = self.block.backward(dy, self.block_params, saved)
        return loss, [grads[k] for k in self.block_params] + [dweight, dbias, dw]

    def reference(self, x, target):
        """Loss and gradients of the current parameters in 64 bits."""
        p = [t.double().requires_grad_() for t in self.params]
        b = dict(zip(self.block_params, p))
        h = torch.nn.functional.layer_norm(x.double(), (H,), b["weight"], b["bias"], EPS)
        z = torch.mm(h, b["w1"]) + b["b1"]
        a = torch.nn.functional.gelu(z, approximate="tanh") if self.act == "gelu_tanh" else torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        y = x.double() + torch.mm(a, b["w2"]) + b["b2"]
        h = torch.nn.functional.layer_norm(y, (H,), p[6], p[7], EPS)
        loss = torch.nn.functional.cross_entropy(torch.mm(h, p[8].t()), target, ignore_index=-100, reduction="none")
        (loss.sum() / (target >= 0).sum()).backward()
        return loss.detach(), [t.grad for t in p]

    def close(self):
        for part in (self.block, self.norm, self.loss, self.clip, self.opt):
            part.close()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,act", [("f16", "gelu_tanh"), ("bf16", "swiglu")])
def test_training_steps(dtype, act, bits):
    """Every step's losses and gradients are those of the parameters that the step before left, its update is AdamW's of
    its own gradients, and the parameters are the master weights rounded."""
    u = torch.finfo({"f16": torch.float16, "bf16": torch.bfloat16}[dtype]).eps / 2
    m = Model(dtype, act, bits)
    g = torch.Generator("cuda").manual_seed(2)
    norm, scale = (torch.empty(1, device="cuda") for _ in range(2))
    for step in range(1, 4):
        x = torch.randn(ROWS, H, generator=g, device="cuda").to(m.params[0].dtype)
        target = torch.randint(V, (ROWS,), generator=g, device="cuda")
        target[torch.rand(ROWS, generator=g, device="cuda") < 0.2] = -100
        ref_loss, ref = m.reference(x, target)
        loss, grads = m.gradients(x, target)
        m.clip.forward(grads, norm, scale, max_norm=0.5, unscale=1 / m.scale_of_loss)
        torch.cuda.synchronize()
        # a chain of some ten roundings of u each, of intermediate values of the results' size
        assert float((loss.double() - ref_loss).norm() / ref_loss.norm()) <= 8 * u
        for got, want in zip(grads, ref):
            assert float((got.double() / m.scale_of_loss - want).norm() / want.norm()) <= 16 * u
        total = math.sqrt(sum(float(t.double().square().sum()) for t in grads)) / m.scale_of_loss
        assert abs(float(norm) - total) <= 1e-6 * total
        assert abs(float(scale) * m.scale_of_loss - min(1.0, 0.5 / total)) <= 1e-6
        before = [t.clone().double() for t in m.opt.master]
        if bits == 32:
            old = [(a.clone().double(), b.clone().double()) for a, b in zip(m.opt.m, m.opt.v)]
        m.opt.step(grads, 1e-2, scale=scale)
        torch.cuda.synchronize()
        assert int(m.opt.t) == step
        for i, (p, master) in enumerate(zip(m.params, m.opt.master)):
            assert torch.equal(p, master.to(p.dtype))
            change = master.double() - before[i] * (1 - 1e-2 * m.opt.decay[i])
            # (AdamW's step is at most lr (1 - b1) / sqrt(1 - b2) / (1 - b1^t) sqrt(1 - b2^t) of a first gradient)
            assert float(change.abs().max()) <= 1e-2 * 4.5
            if bits == 32:
                gr = grads[i].double() * float(scale)
                m1, v1 = 0.9 * old[i][0] + 0.1 * gr, 0.95 * old[i][1] + 0.05 * gr * gr
                want = -1e-2 * (m1 / (1 - 0.9 ** step)) / (torch.sqrt(v1 / (1 - 0.95 ** step)) + 1e-8)
                # (roundings of weights about a hundred times the change to fp32: 2^-24 100, and the states')
                assert float((change - want).norm() / want.norm()) <= 1e-4
    m.close()


def test_a_step_that_overflows_is_left_out():
    """An infinite loss scale gives gradients that are not finite: the scale is NaN, and nothing changes."""
    m = Model("f16", "gelu_tanh", 8)
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(ROWS, H, generator=g, device="cuda").half()
    target = torch.randint(V, (ROWS,), generator=g, device="cuda")
    m.scale_of_loss = 2.0 ** 30
    norm, scale = (torch.empty(1, device="cuda") for _ in range(2))
    _, grads = m.gradients(x, target)
    m.clip.forward(grads, norm, scale, max_norm=1.0, unscale=2.0 ** -30)
    before = [t.clone() for t in m.params + m.opt.master + m.opt.m + m.opt.v]
    m.opt.step(grads, 1e-2, scale=scale)
    torch.cuda.synchronize()
    assert math.isnan(float(scale)) and int(m.opt.t) == 0
    for a, b in zip(m.params + m.opt.master + m.opt.m + m.opt.v, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    m.close()
