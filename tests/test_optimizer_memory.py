"""An optimizer's tensors share no memory: a step writes all of them at once (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd.mlp_train import _check_apart


def pieces(*sizes, dtype=torch.float32):
    """Neighbouring views of one buffer."""
    return list(torch.zeros(sum(sizes), dtype=dtype).split(sizes))


def test_neighbours_are_apart():
    a, b = pieces(5, 0, 7, 256), pieces(5, 0, 7, 256, dtype=torch.uint8)
    _check_apart([("m", a), ("v", b), ("step", [torch.zeros(1, dtype=torch.int64)])])
    _check_apart([("m", []), ("v", [torch.zeros(0)] * 3)])


@pytest.mark.parametrize("change", [lambda m, v: (m[:1] * 3, v),                        # one tensor for all
                                    lambda m, v: (m, [v[0], m[1], v[2]]),               # m and v the same
                                    lambda m, v: (m, [v[0], v[1], m[2][3:4]]),          # a part of another one
                                    lambda m, v: ([m[0], m[1], torch.as_strided(m[2], (8,), (1,), m[2].storage_offset() - 1)], v)])
def test_shared_memory_is_refused(change):
    m, v = change(pieces(8, 8, 8), pieces(8, 8, 8))
    with pytest.raises(ValueError, match="share memory"):
        _check_apart([("m", m), ("v", v)])


def test_the_message_names_both():
    t = torch.zeros(8)
    with pytest.raises(ValueError, match=r"master\[0\] and m\[1\] share memory"):
        _check_apart([("master", [t]), ("m", [torch.zeros(3), t[7:]])])
