"""The training step's C ABI without a GPU: every symbol of include/mlp_train.h is exported and bound, and the argument
checks that need no device refuse what they should with a message."""
import ctypes
import os
import re

import pytest

from consumer_gemm_chain_amd import mlp_chain as mc
from consumer_gemm_chain_amd import mlp_train as mt

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_declared_symbol_is_exported_and_bound():
    text = open(os.path.join(ROOT, "include", "mlp_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    syms = set(re.findall(r"\b(mlp_(?:loss|grad_norm|adamw)_\w+)\s*\(", text))
    assert syms == set(mt.EXPORTS)
    lib = ctypes.CDLL(mc.LIB_PATH)
    for s in syms:
        assert hasattr(lib, s), s
        assert callable(getattr(mt, s)), s


@pytest.mark.parametrize("args,needle", [
    ((0, 64, 100, 0), "sizes"),
    (((1 << 24) + 1, 64, 100, 0), "sizes"),
    ((4, 0, 100, 0), "sizes"),
    ((4, 60, 100, 0), "multiple of 8"),
    ((4, 1 << 22, 100, 0), "sizes"),
    ((4, 64, 0, 0), "sizes"),
    ((4, 64, 1 << 22, 0), "sizes"),
    ((1 << 24, 64, 1 << 15, 0), "2\\^38"),
    ((1 << 24, 1 << 15, 64, 0), "2\\^38"),
    ((4, 1 << 20, 1 << 20, 0), "2\\^38"),
    ((4, 64, 100, 2), "dtype"),
])
def test_loss_create_refuses(args, needle):
    with pytest.raises(mc.MlpChainError, match=needle):
        mt.mlp_loss_create(*args)


def test_grad_norm_create_refuses():
    with pytest.raises(mc.MlpChainError, match="dtype"):
        mt.mlp_grad_norm_create(2)


@pytest.mark.parametrize("args,needle", [
    ((2, 32, 0.9, 0.99, 1e-8, 0), "dtype"),
    ((0, 16, 0.9, 0.99, 1e-8, 0), "32 or 8 bits"),
    ((0, 32, 1.0, 0.99, 1e-8, 0), "beta"),
    ((0, 32, -0.1, 0.99, 1e-8, 0), "beta"),
    ((0, 32, 0.9, 1.0, 1e-8, 0), "beta"),
    ((0, 32, 0.9, float("nan"), 1e-8, 0), "beta"),
    ((0, 32, 0.9, 0.99, -1e-8, 0), "eps"),
    ((0, 32, 0.9, 0.99, float("inf"), 0), "eps"),
])
def test_adamw_create_refuses(args, needle):
    with pytest.raises(mc.MlpChainError, match=needle):
        mt.mlp_adamw_create(*args)


def test_null_handles():
    lib = mt._library()
    assert lib.mlp_loss_forward(None, 1, None, 8, None, 8, None, None, None, None) == mc.MLP_EINVAL
    assert lib.mlp_loss_backward(None, 1, None, 8, None, 8, *[None] * 5, 8, None, 8, None) == mc.MLP_EINVAL
    assert lib.mlp_loss_debug_set_plan(None, 0, 0, 0) == mc.MLP_EINVAL
    assert lib.mlp_grad_norm_forward(None, 0, None, None, 1.0, 1.0, None, None, None) == mc.MLP_EINVAL
    assert lib.mlp_adamw_step(None, 0, None, None, 1.0, None, None, None, None) == mc.MLP_EINVAL
    for destroy in (lib.mlp_loss_destroy, lib.mlp_grad_norm_destroy, lib.mlp_adamw_destroy):
        assert destroy(None) == mc.MLP_OK
