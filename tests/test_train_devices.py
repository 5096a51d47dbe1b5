"""Operands on another device than the handle's are refused before a kernel could read them (no GPU needed: the
tensors are stand-ins)."""
import pytest

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpAdamW, MlpGradNorm, MlpLoss
from tests.test_block_devices import On


def loss_layer():
    """A loss whose handle is on device 1, without its handle: a call that passes the checks is refused for that."""
    t = MlpLoss.__new__(MlpLoss)
    t._set_type("f16")
    t._i64, t.device = torch.int64, 1
    t.rows, t.H, t.V = 4, 64, 100
    return t


@pytest.mark.parametrize("wrong", [0, 2, -1])
def test_loss_operands_on_another_device_are_refused(wrong):
    f32 = torch.float32
    base = {"x": ((4, 64), torch.float16), "w": ((100, 64), torch.float16), "target": ((4,), torch.int64),
            "loss": ((4,), f32), "lse": ((4,), f32)}
    more = {"dloss": ((4,), f32), "dlse": ((4,), f32), "dx": ((4, 64), torch.float16), "dw": ((100, 64), torch.float16)}
    make = lambda spec, bad: {k: On(wrong if k == bad else 1, *s, dtype=d) for k, (s, d) in spec.items()}  # noqa: E731
    layer = loss_layer()
    for bad in base:
        with pytest.raises(ValueError, match="device"):
            layer.forward(stream=0, **make(base, bad))
    back = {k: v for k, v in base.items() if k != "loss"} | more
    for bad in back:
        with pytest.raises(ValueError, match="device"):
            layer.backward(stream=0, **make(back, bad))


def test_optimizer_tensors_on_another_device_are_refused():
    """Tensors of the host and of a device that a handle on device 1 is not for."""
    norm = MlpGradNorm.__new__(MlpGradNorm)
    norm._set_type("f16")
    norm.device = 1
    for where in ("cpu", "meta"):
        with pytest.raises(ValueError, match="device 1"):
            norm.forward([torch.empty(4, dtype=torch.float16, device=where)], On(1, 1, dtype=torch.float32), stream=0)
    opt = MlpAdamW.__new__(MlpAdamW)
    opt._set_type("f16")
    opt.device, opt.params, opt._params, opt._shapes, opt._table = 1, [], [], [torch.Size((4,))], None
    with pytest.raises(ValueError, match="device 1"):
        opt.step([torch.empty(4, dtype=torch.float16)], 1e-3, stream=0)
