"""Thin Python binding of the C ABI in include/mlp_block.h (ctypes): layer
norm and the linear layer of a transformer MLP block, forward and backward,
and the whole pre-norm block composed of them.

As in the chain's binding, only argument marshalling happens here; torch
supplies device memory and streams, and there is no fallback.
"""
from __future__ import annotations

import ctypes

from .mlp_chain import ACTS, DTYPES, MLP_EINVAL, MlpChainError, _check, load_library, mlp_chain_last_error

EXPORTS = ("mlp_norm_create", "mlp_norm_forward", "mlp_norm_backward", "mlp_norm_destroy",
           "mlp_linear_create", "mlp_linear_forward", "mlp_linear_backward", "mlp_linear_destroy",
           "mlp_linear_plan", "mlp_linear_debug_set_plan")

PLAN_FIELDS = ("config", "S", "BM", "BN", "Mt", "Nt", "ksp", "part_bytes", "direct")

_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        vp, i64, ci, f = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        lib.mlp_norm_create.argtypes = [i64, ci, f, ci]
        lib.mlp_norm_create.restype = vp
        lib.mlp_norm_forward.argtypes = [vp, i64, vp, i64, vp, vp, vp, i64, vp, vp, vp]
        lib.mlp_norm_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp]
        lib.mlp_linear_create.argtypes = [i64, i64, i64, ci, ci, ci]
        lib.mlp_linear_create.restype = vp
        lib.mlp_linear_forward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp]
        lib.mlp_linear_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, vp]
        lib.mlp_linear_plan.argtypes = [i64, i64, i64, ci, ci, ci, ctypes.POINTER(i64), ci]
        lib.mlp_linear_debug_set_plan.argtypes = [vp, ci, ci, ci]
        for name in ("mlp_norm_destroy", "mlp_linear_destroy"):
            getattr(lib, name).argtypes = [vp]
        for name in EXPORTS:
            if not name.endswith("_create"):
                getattr(lib, name).restype = ci
        _lib = lib
    return _lib


# ---- the C ABI, name for name (pointers are integers, NULL is None) ------------

def _created(h):
    if not h:
        raise MlpChainError(MLP_EINVAL, mlp_chain_last_error())
    return h


def mlp_norm_create(H: int, dtype: int, eps: float, grad: bool = True) -> int:
    return _created(_library().mlp_norm_create(int(H), int(dtype), float(eps), int(bool(grad))))


def mlp_norm_forward(h, rows, x, ldx, weight, bias, y, ldy, mean, rstd, hip_stream) -> int:
    return _check(_library().mlp_norm_forward(h, rows, x, ldx, weight, bias, y, ldy, mean, rstd, hip_stream))


def mlp_norm_backward(h, rows, dy, lddy, x, ldx, weight, mean, rstd, dres, lddres, dx, lddx, dweight, dbias,
                      hip_stream) -> int:
    return _check(_library().mlp_norm_backward(h, rows, dy, lddy, x, ldx, weight, mean, rstd, dres, lddres, dx, lddx,
                                               dweight, dbias, hip_stream))


def mlp_norm_destroy(h: int | None) -> int:
    return _check(_library().mlp_norm_destroy(h))


def mlp_linear_create(max_rows: int, K: int, N: int, act: int, dtype: int, grad: bool = True) -> int:
    return _created(_library().mlp_linear_create(int(max_rows), int(K), int(N), int(act), int(dtype), int(bool(grad))))


def mlp_linear_forward(h, rows, x, ldx, w, ldw, bias, residual, ldres, y, ldy, z, ldz, hip_stream) -> int:
    return _check(_library().mlp_linear_forward(h, rows, x, ldx, w, ldw, bias, residual, ldres, y, ldy, z, ldz,
                                                hip_stream))


def mlp_linear_backward(h, rows, dy, lddy, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db, hip_stream) -> int:
    return _check(_library().mlp_linear_backward(h, rows, dy, lddy, x, ldx, w, ldw, z, ldz, dx, lddx, dw, lddw, db,
                                                 hip_stream))


def mlp_linear_destroy(h: int | None) -> int:
    return _check(_library().mlp_linear_destroy(h))


def mlp_linear_plan(rows: int, K: int, N: int, act: int, op: int, cus: int) -> dict:
    """The plan of pass `op` (0: x W, 1: dz W^T alone, 2: x^T dz alone, 3 and 4: dz W^T and x^T dz in one
    launch) on a GPU with `cus` CUs (host only)."""
    arr = (ctypes.c_int64 * len(PLAN_FIELDS))()
    _check(_library().mlp_linear_plan(int(rows), int(K), int(N), int(act), int(op), int(cus), arr, len(PLAN_FIELDS)))
    return dict(zip(PLAN_FIELDS, (int(v) for v in arr)))


def mlp_linear_debug_set_plan(h: int, op: int, config_id: int, split: int) -> int:
    return _check(_library().mlp_linear_debug_set_plan(h, int(op), int(config_id), int(split)))


# ---- convenience wrappers over torch tensors ------------------------------------

class _Layer:
    """Owns one handle; `_destroy` releases it.  The checks below run on every
    call, beside a few microseconds of kernel, and touch each tensor little."""
    h = None
    device = None       # the handle's: the current one when it was created

    def _set_type(self, dtype: str):
        import torch
        self.dtype = dtype
        self.torch_dtype = torch.float16 if dtype == "f16" else torch.bfloat16
        self._f32 = torch.float32
        # the current stream's handle without building a Stream object (2.7 us of a call)
        self._raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda device: torch.cuda.current_stream(device).cuda_stream)

    def close(self):
        h, self.h = self.h, None
        if h:
            self._destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def _stream(self, stream, t):
        """The handle of `stream`, or of the current stream of t's device."""
        if stream is not None:
            return int(getattr(stream, "cuda_stream", stream))
        return self._raw_stream(t.get_device())

    def _hold(self, h):
        import torch
        self.h, self.device = h, torch.cuda.current_device()

    def _rows(self, name, t, rows, width):
        """Pointer and row stride of a [rows, width] operand (None, 0: absent)."""
        if t is None:
            return None, 0
        if t.shape != (rows, width):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, width)}")
        if t.dtype != self.torch_dtype or t.get_device() != self.device:
            raise ValueError(f"{name} must be a {self.dtype} tensor on the handle's device {self.device}")
        ld, unit = t.stride()
        if unit != 1 and width > 1:
            raise ValueError(f"{name} must have contiguous rows, got strides {(ld, unit)}")
        return t.data_ptr(), ld if rows > 1 else width      # (a single row's stride is never used)

    def _vector(self, name, t, n, dtype):
        """Pointer of a contiguous vector (None: absent)."""
        if t is None:
            return None
        if t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous vector of {n} elements, got shape {tuple(t.shape)}")
        if t.dtype != dtype or t.get_device() != self.device:
            raise ValueError(f"{name} must be a {dtype} tensor on the handle's device {self.device}")
        return t.data_ptr()


class MlpNorm(_Layer):
    """Layer norm over rows of H elements, on the device that is current when it
    is made.  Outputs are the caller's tensors; work is enqueued on the current
    stream of that device (or `stream`).  With
    grad=False the handle holds no workspace and only runs forward."""

    def __init__(self, H: int, dtype: str = "f16", eps: float = 1e-5, grad: bool = True):
        self.H, self.eps = int(H), float(eps)
        self._set_type(dtype)
        self._hold(mlp_norm_create(H, DTYPES[dtype], eps, grad))

    _destroy = staticmethod(mlp_norm_destroy)

    def forward(self, x, weight, bias, out, mean=None, rstd=None, stream=None):
        """out = norm(x) weight + bias ([rows, H]); `mean` and `rstd` (float32
        [rows]) receive the statistics the gradient needs."""
        rows, H, dt, f32 = x.shape[0], self.H, self.torch_dtype, self._f32
        px, ldx = self._rows("x", x, rows, H)
        py, ldy = self._rows("out", out, rows, H)
        mlp_norm_forward(self.h, rows, px, ldx, self._vector("weight", weight, H, dt),
                         self._vector("bias", bias, H, dt), py, ldy, self._vector("mean", mean, rows, f32),
                         self._vector("rstd", rstd, rows, f32), self._stream(stream, x))
        return out

    def backward(self, dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, dres=None, stream=None):
        """The gradients of `forward`; `dres` is added to dx."""
        rows, H, dt, f32 = x.shape[0], self.H, self.torch_dtype, self._f32
        pdy, lddy = self._rows("dy", dy, rows, H)
        px, ldx = self._rows("x", x, rows, H)
        pr, ldr = self._rows("dres", dres, rows, H)
        pdx, lddx = self._rows("dx", dx, rows, H)
        mlp_norm_backward(self.h, rows, pdy, lddy, px, ldx, self._vector("weight", weight, H, dt),
                          self._vector("mean", mean, rows, f32), self._vector("rstd", rstd, rows, f32), pr, ldr, pdx,
                          lddx, self._vector("dweight", dweight, H, dt), self._vector("dbias", dbias, H, dt),
                          self._stream(stream, x))
        return dx


class MlpLinear(_Layer):
    """Linear layer K -> N with bias, activation and residual for calls of up
    to `rows` rows.  W is [K, gN] (g = 2 for swiglu: gate, then up) and given
    with every call: one handle serves all layers of its sizes.  With
    grad=False it only runs forward and holds less."""

    def __init__(self, rows: int, K: int, N: int, act: str = "none", dtype: str = "f16", grad: bool = True):
        self.rows, self.K, self.N, self.act = int(rows), int(K), int(N), act
        self.gN = self.N * (2 if act == "swiglu" else 1)
        self._set_type(dtype)
        self._hold(mlp_linear_create(rows, K, N, ACTS[act], DTYPES[dtype], grad))

    _destroy = staticmethod(mlp_linear_destroy)

    def forward(self, x, w, out, bias=None, residual=None, z=None, stream=None):
        """out = act(x w + bias) + residual; `z` receives x w + bias."""
        rows = x.shape[0]
        px, ldx = self._rows("x", x, rows, self.K)
        pw, ldw = self._rows("w", w, self.K, self.gN)
        pr, ldr = self._rows("residual", residual, rows, self.N)
        py, ldy = self._rows("out", out, rows, self.N)
        pz, ldz = self._rows("z", z, rows, self.gN)
        mlp_linear_forward(self.h, rows, px, ldx, pw, ldw, self._vector("bias", bias, self.gN, self.torch_dtype), pr,
                           ldr, py, ldy, pz, ldz, self._stream(stream, x))
        return out

    def backward(self, dy, x, w, dx=None, dw=None, db=None, z=None, stream=None):
        """The gradients of `forward` that are asked for; activations need the
        saved `z`.  The residual's gradient is dy itself."""
        rows = dy.shape[0]
        pdy, lddy = self._rows("dy", dy, rows, self.N)
        px, ldx = self._rows("x", x, rows, self.K)
        pw, ldw = self._rows("w", w, self.K, self.gN)
        pz, ldz = self._rows("z", z, rows, self.gN)
        pdx, lddx = self._rows("dx", dx, rows, self.K)
        pdw, lddw = self._rows("dw", dw, self.K, self.gN)
        mlp_linear_backward(self.h, rows, pdy, lddy, px, ldx, pw, ldw, pz, ldz, pdx, lddx, pdw, lddw,
                            self._vector("db", db, self.gN, self.torch_dtype), self._stream(stream, dy))
        return dx, dw, db


class MlpBlock:
    """The pre-norm MLP block y = x + act(norm(x) W1 + b1) W2 + b2 for up to
    `rows` rows, H wide with I inner columns: one norm and two linear layers,
    and their gradients.  `params` maps names to tensors: weight, bias [H],
    w1 [H, gI], b1 [gI], w2 [I, H], b2 [H]; None leaves out the norm's scale or
    shift or a bias.  grad=False: forward only."""

    def __init__(self, rows: int, H: int, I: int, act: str = "gelu_tanh", dtype: str = "f16", eps: float = 1e-5,
                 grad: bool = True):
        self.H, self.I, self.act, self.dtype = int(H), int(I), act, dtype
        self.norm = MlpNorm(H, dtype, eps, grad)
        self.lin1 = MlpLinear(rows, H, I, act, dtype, grad)
        self.lin2 = MlpLinear(rows, I, H, "none", dtype, grad)

    def close(self):
        for layer in (self.norm, self.lin1, self.lin2):
            layer.close()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def forward(self, x, params, save: bool = False):
        """Returns y, and with `save` also what `backward` needs."""
        import torch
        rows, gI = x.shape[0], self.lin1.gN
        n, a, y = torch.empty_like(x), x.new_empty(rows, self.I), torch.empty_like(x)
        mean = rstd = z = None
        if save:
            mean, rstd = (torch.empty(rows, dtype=torch.float32, device=x.device) for _ in range(2))
            z = x.new_empty(rows, gI) if self.act != "none" else None
        self.norm.forward(x, params["weight"], params["bias"], n, mean, rstd)
        self.lin1.forward(n, params["w1"], a, bias=params["b1"], z=z)
        self.lin2.forward(a, params["w2"], y, bias=params["b2"], residual=x)
        return (y, (x, n, a, z, mean, rstd)) if save else y

    def backward(self, dy, params, saved):
        """dx and the gradients of every parameter, by name (None for an absent one)."""
        import torch
        x, n, a, z, mean, rstd = saved
        grads = {k: None if v is None else torch.empty_like(v) for k, v in params.items()}
        da, dn, dx = torch.empty_like(a), torch.empty_like(n), torch.empty_like(x)
        self.lin2.backward(dy, a, params["w2"], dx=da, dw=grads["w2"], db=grads["b2"])
        self.lin1.backward(da, n, params["w1"], dx=dn, dw=grads["w1"], db=grads["b1"], z=z)
        self.norm.backward(dn, x, params["weight"], mean, rstd, dx, grads["weight"], grads["bias"], dres=dy)
        return dx, grads
