"""The whole block without biases, scale or shift on the GPU."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpBlock  # noqa: E402
from tests.test_block_gpu import DT, EPS, U, act_ref, block_params, gen, norm_ref  # noqa: E402


@pytest.mark.parametrize("absent", [("b1", "b2"), ("weight", "bias", "b1", "b2"), ("bias", "b1")])
@pytest.mark.parametrize("rows,H,I,act,dtype", [(130, 520, 264, "swiglu", "bf16"), (20, 512, 2048, "gelu_tanh", "f16")])
def test_block_without_some_parameters(rows, H, I, act, dtype, absent):
    """Forward and gradients against 64-bit autograd, within the four roundings of the block's own test."""
    p = {**block_params(H, I, act, dtype), **dict.fromkeys(absent)}
    n = gen(43)
    x, dy = n(rows, H).to(DT[dtype]), (0.1 * n(rows, H)).to(DT[dtype])
    with MlpBlock(rows, H, I, act, dtype, EPS) as block:
        y, saved = block.forward(x, p, save=True)
        dx, grads = block.backward(dy, p, saved)
        torch.cuda.synchronize()
    q = {k: None if v is None else v.double().requires_grad_() for k, v in p.items()}
    xd = x.double().requires_grad_()
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    plus = lambda t: zero if t is None else t  # noqa: E731
    h = torch.mm(norm_ref(xd, q["weight"], q["bias"])[0], q["w1"]) + plus(q["b1"])
    ref = xd + torch.mm(act_ref(h, act, I), q["w2"]) + plus(q["b2"])
    ref.backward(dy.double())
    checks = [("y", y, ref.detach()), ("dx", dx, xd.grad)]
    checks += [(k, grads[k], q[k].grad) for k in p if p[k] is not None]
    for name, got, want in checks:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 4 * U[dtype], (name, rel)
    assert all(grads[k] is None for k in absent)
