"""The block operators' C ABI without a GPU: every symbol of
include/mlp_block.h is exported and bound, and the argument checks that need
no device refuse what they should with a message."""
import ctypes
import os
import re

import pytest

from consumer_gemm_chain_amd import mlp_block as mb
from consumer_gemm_chain_amd import mlp_chain as mc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_declared_symbol_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "mlp_block.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    syms = set(re.findall(r"\b(mlp_(?:norm|linear)_\w+)\s*\(", text))
    assert syms == set(mb.EXPORTS)
    lib = ctypes.CDLL(mc.LIB_PATH)
    for s in syms:
        assert hasattr(lib, s), s
        assert callable(getattr(mb, s)), s


@pytest.mark.parametrize("args,needle", [
    ((0, 0, 1e-5), "H must be"),
    (((1 << 22) + 1, 0, 1e-5), "H must be"),
    ((64, 2, 1e-5), "dtype"),
    ((64, 0, -1.0), "eps"),
    ((64, 0, float("nan")), "eps"),
    ((64, 0, float("inf")), "eps"),
])
def test_norm_create_refuses(args, needle):
    with pytest.raises(mc.MlpChainError, match=needle):
        mb.mlp_norm_create(*args)


@pytest.mark.parametrize("args,needle", [
    ((0, 64, 64, 0, 0), "sizes"),
    (((1 << 24) + 1, 64, 64, 0, 0), "sizes"),
    ((4, 0, 64, 0, 0), "sizes"),
    ((4, 64, 1 << 22, 0, 0), "sizes"),
    ((4, 60, 64, 0, 0), "multiples of 8"),
    ((4, 64, 36, 0, 0), "multiples of 8"),
    ((4, 64, 64, 3, 0), "activation"),
    ((4, 64, 64, -1, 0), "activation"),
    ((4, 64, 64, 0, 2), "dtype"),
])
def test_linear_create_refuses(args, needle):
    with pytest.raises(mc.MlpChainError, match=needle):
        mb.mlp_linear_create(*args)


def test_null_handles():
    lib = mb._library()
    assert lib.mlp_norm_forward(None, 1, None, 8, None, None, None, 8, None, None, None) == mc.MLP_EINVAL
    assert lib.mlp_norm_backward(*[None, 1] + [None, 8] * 2 + [None] * 3 + [None, 8] * 2 + [None] * 3) == mc.MLP_EINVAL
    assert lib.mlp_linear_forward(None, 1, None, 8, None, 8, None, None, 8, None, 8, None, 8, None) == mc.MLP_EINVAL
    assert lib.mlp_linear_backward(*[None, 1] + [None, 8] * 6 + [None] * 2) == mc.MLP_EINVAL
    assert lib.mlp_norm_destroy(None) == mc.MLP_OK
    assert lib.mlp_linear_destroy(None) == mc.MLP_OK
