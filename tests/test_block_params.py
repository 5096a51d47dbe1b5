"""The whole block's parameters without a GPU: what its gradient asks of the layers, which are stand-ins here."""
import pytest

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpBlock


class Layer:
    """Takes a call of a layer and marks the gradients it is given."""

    def __init__(self, gN=None):
        self.gN = gN

    def close(self):
        pass

    def forward(self, *args, **kw):
        pass

    def backward(self, *args, **kw):
        for t in (*args[5:], kw.get("dx"), kw.get("dw"), kw.get("db")):
            if t is not None:
                t.fill_(1)


@pytest.mark.parametrize("absent", [(), ("b1", "b2"), ("weight", "bias", "b1", "b2"), ("bias",)])
def test_gradients_of_absent_parameters_are_none(absent):
    rows, H, I = 3, 16, 24
    block = MlpBlock.__new__(MlpBlock)
    block.H, block.I, block.act, block.dtype = H, I, "swiglu", "f16"
    block.norm, block.lin1, block.lin2 = Layer(), Layer(2 * I), Layer(H)
    p = {"weight": torch.ones(H), "bias": torch.ones(H), "w1": torch.ones(H, 2 * I), "b1": torch.ones(2 * I),
         "w2": torch.ones(I, H), "b2": torch.ones(H)}
    p.update(dict.fromkeys(absent))
    x = torch.ones(rows, H)
    _, saved = block.forward(x, p, save=True)
    dx, grads = block.backward(x, p, saved)
    assert set(grads) == set(p) and dx.shape == x.shape
    for k, v in p.items():
        assert (grads[k] is None) if v is None else (grads[k].shape == v.shape), k
