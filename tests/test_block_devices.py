"""Operands on another device than the handle's are refused before a kernel could read them (no GPU needed: the
tensors are stand-ins)."""
import pytest

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpLinear, MlpNorm


class On:
    """What the checks look at of a contiguous fp16 or fp32 tensor on `device` (-1: the host)."""

    def __init__(self, device, *shape, dtype=torch.float16):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device
        self.is_cuda = device >= 0

    def get_device(self):
        return self.device_index

    def stride(self):
        return (self.shape[-1], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


def layer(kind):
    """A layer whose handle is on device 1, without its handle: a call that passes the checks is refused for that."""
    t = kind.__new__(kind)
    t._set_type("f16")
    t.device = 1
    t.H, t.rows, t.K, t.N, t.gN, t.act = 64, 4, 64, 64, 64, "none"
    return t


@pytest.mark.parametrize("wrong", [0, 2, -1])
def test_operands_on_another_device_are_refused(wrong):
    norm, lin = layer(MlpNorm), layer(MlpLinear)
    m, v = On(1, 4, 64), On(1, 64)
    w = On(1, 64, 64)
    for operand in range(6):
        a = [m, v, v, m, On(1, 4, dtype=torch.float32), On(1, 4, dtype=torch.float32)]
        a[operand] = On(wrong, *a[operand].shape, dtype=a[operand].dtype)
        with pytest.raises(ValueError, match="device"):
            norm.forward(*a, stream=0)
    for operand in ("x", "w", "out", "bias", "residual", "z"):
        k = {"x": m, "w": w, "out": m, "bias": v, "residual": m, "z": m}
        k[operand] = On(wrong, *k[operand].shape)
        with pytest.raises(ValueError, match="device"):
            lin.forward(stream=0, **k)
