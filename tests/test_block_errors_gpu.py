"""What the block operators make of errors on the GPU: their own and those that other calls of the thread left."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from consumer_gemm_chain_amd import MlpChainError, MlpLinear, MlpNorm  # noqa: E402
from consumer_gemm_chain_amd import mlp_chain as mc  # noqa: E402

OUT_OF_MEMORY = 2       # hipErrorOutOfMemory


@pytest.fixture
def runtime():
    """The HIP runtime that the library calls; the thread's last error is cleared around the test."""
    hip = ctypes.CDLL(mc.LIB_PATH)
    hip.hipMalloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_size_t]
    hip.hipGetLastError()
    yield hip
    hip.hipGetLastError()


def test_an_error_left_by_another_call_is_not_reported(runtime):
    """An allocation of the caller's own fails; every launch after it succeeds, and the error stays the caller's."""
    half = lambda *shape: torch.ones(shape, dtype=torch.float16, device="cuda")  # noqa: E731
    f32 = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    x, v, wide, w, dy = half(200, 64), half(64), half(40, 20000), half(64, 24), half(200, 24)
    s, s40 = f32(200), f32(40)
    nx, ny, nw, nb = half(200, 64), half(200, 64), half(64), half(64)
    lx, lw, lb, ly = half(200, 64), half(64, 24), half(24), half(200, 24)
    wy, wx, ww = half(40, 20000), half(40, 20000), half(20000)
    p = ctypes.c_void_p()
    with MlpNorm(64) as norm, MlpNorm(20000) as sweep, MlpLinear(200, 64, 24, "gelu_tanh") as lin:
        torch.cuda.synchronize()
        # (torch's own launches would report it: everything they make is made above)
        assert runtime.hipMalloc(ctypes.byref(p), 1 << 50) == OUT_OF_MEMORY
        norm.forward(x, v, v, ny)
        norm.backward(x, x, v, s, s, nx, nw, nb)
        norm.backward(x[:3], x[:3], v, s[:3], s[:3], nx[:3], nw, nb)
        sweep.forward(wide, None, None, wy)
        sweep.backward(wide, wide, None, s40, s40, wx, ww)
        lin.forward(x, w, ly)
        lin.backward(dy, x, w, dx=lx, dw=lw, db=lb, z=dy)
        lin.backward(dy, None, w, dx=lx, z=dy)
        lin.backward(dy, x, None, dw=lw, db=lb, z=dy)
        assert runtime.hipGetLastError() == OUT_OF_MEMORY
        torch.cuda.synchronize()


def test_a_handle_that_does_not_fit_leaves_no_error(runtime):
    """create refuses, and torch's next launch does not find the failed allocation."""
    with pytest.raises(MlpChainError, match="hipMalloc"):
        MlpLinear(1 << 24, 8, 1 << 21, "gelu_tanh")
    assert runtime.hipGetLastError() == 0
    with pytest.raises(MlpChainError, match="hipMalloc"):
        MlpLinear(1 << 24, 8, 1 << 21, "gelu_tanh")
    assert bool((torch.ones(8, device="cuda") + 1 == 2).all())
