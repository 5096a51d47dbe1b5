"""Thin Python binding of the C ABI in include/mlp_train.h (ctypes): the
cross entropy of a vocabulary head, the norm of all gradients and AdamW.

As in the other bindings, only argument marshalling happens here; torch
supplies device memory and streams, and there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import math

from .mlp_block import _created, _Layer
from .mlp_chain import DTYPES, _check, load_library

EXPORTS = ("mlp_loss_create", "mlp_loss_forward", "mlp_loss_backward", "mlp_loss_destroy", "mlp_loss_debug_set_plan",
           "mlp_grad_norm_create", "mlp_grad_norm_forward", "mlp_grad_norm_destroy",
           "mlp_adamw_create", "mlp_adamw_step", "mlp_adamw_destroy")

BLOCK = 256         # elements that share a scale in 8-bit states


class AdamwTensor(ctypes.Structure):
    """mlp_adamw_tensor."""
    _fields_ = [("n", ctypes.c_int64), ("w", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("decay", ctypes.c_double)]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        vp, i64, ci, d = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double
        lib.mlp_loss_create.argtypes = [i64, i64, i64, ci, ci]
        lib.mlp_loss_forward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp]
        lib.mlp_loss_backward.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, i64, vp]
        lib.mlp_loss_debug_set_plan.argtypes = [vp, ci, ci, ci]
        lib.mlp_grad_norm_create.argtypes = [ci]
        lib.mlp_grad_norm_forward.argtypes = [vp, i64, vp, vp, d, d, vp, vp, vp]
        lib.mlp_adamw_create.argtypes = [ci, ci, d, d, d, ctypes.c_uint32]
        lib.mlp_adamw_step.argtypes = [vp, i64, vp, vp, d, vp, vp, vp, vp]
        for name in ("mlp_loss_destroy", "mlp_grad_norm_destroy", "mlp_adamw_destroy"):
            getattr(lib, name).argtypes = [vp]
        for name in EXPORTS:
            getattr(lib, name).restype = vp if name.endswith("_create") else ci
        _lib = lib
    return _lib


# ---- the C ABI, name for name (pointers are integers, NULL is None) ------------

def mlp_loss_create(max_rows: int, H: int, V: int, dtype: int, grad: bool = True) -> int:
    return _created(_library().mlp_loss_create(int(max_rows), int(H), int(V), int(dtype), int(bool(grad))))


def mlp_loss_forward(h, rows, x, ldx, w, ldw, target, loss, lse, hip_stream) -> int:
    return _check(_library().mlp_loss_forward(h, rows, x, ldx, w, ldw, target, loss, lse, hip_stream))


def mlp_loss_backward(h, rows, x, ldx, w, ldw, target, lse, dloss, dlse, dx, lddx, dw, lddw, hip_stream) -> int:
    return _check(_library().mlp_loss_backward(h, rows, x, ldx, w, ldw, target, lse, dloss, dlse, dx, lddx, dw, lddw,
                                               hip_stream))


def mlp_loss_destroy(h: int | None) -> int:
    return _check(_library().mlp_loss_destroy(h))


def mlp_loss_debug_set_plan(h: int, product: int, config_id: int, split: int) -> int:
    return _check(_library().mlp_loss_debug_set_plan(h, int(product), int(config_id), int(split)))


def mlp_grad_norm_create(dtype: int) -> int:
    return _created(_library().mlp_grad_norm_create(int(dtype)))


def mlp_grad_norm_forward(h, count, sizes, grads, unscale, max_norm, norm, scale, hip_stream) -> int:
    """`sizes` and `grads`: ctypes arrays of `count` int64 and pointers."""
    return _check(_library().mlp_grad_norm_forward(h, count, sizes, grads, unscale, max_norm, norm, scale, hip_stream))


def mlp_grad_norm_destroy(h: int | None) -> int:
    return _check(_library().mlp_grad_norm_destroy(h))


def mlp_adamw_create(dtype: int, bits: int, beta1: float, beta2: float, eps: float, seed: int) -> int:
    return _created(_library().mlp_adamw_create(int(dtype), int(bits), float(beta1), float(beta2), float(eps),
                                                int(seed) & 0xFFFFFFFF))


def mlp_adamw_step(h, count, tensors, grads, lr, lr_scale, scale, t, hip_stream) -> int:
    """`tensors` and `grads`: ctypes arrays of `count` AdamwTensor and pointers."""
    return _check(_library().mlp_adamw_step(h, count, tensors, grads, lr, lr_scale, scale, t, hip_stream))


def mlp_adamw_destroy(h: int | None) -> int:
    return _check(_library().mlp_adamw_destroy(h))


# ---- convenience wrappers over torch tensors ------------------------------------

class MlpLoss(_Layer):
    """Softmax cross entropy over V words from H-wide rows, for calls of up to
    `rows` rows: z = x W^T with W [V, H] (an embedding's layout), without
    keeping z.  W is given with every call.  Rows with a negative target are
    left out.  With grad=False it only runs forward and holds less."""

    def __init__(self, rows: int, H: int, V: int, dtype: str = "f16", grad: bool = True):
        import torch
        self.rows, self.H, self.V = int(rows), int(H), int(V)
        self._set_type(dtype)
        self._i64 = torch.int64
        self._hold(mlp_loss_create(rows, H, V, DTYPES[dtype], grad))

    _destroy = staticmethod(mlp_loss_destroy)

    def forward(self, x, w, target, loss, lse, stream=None):
        """loss and lse (float32 [rows]) of x [rows, H] and target (int64 [rows]); loss may be None."""
        rows, f32 = x.shape[0], self._f32
        px, ldx = self._rows("x", x, rows, self.H)
        pw, ldw = self._rows("w", w, self.V, self.H)
        mlp_loss_forward(self.h, rows, px, ldx, pw, ldw, self._vector("target", target, rows, self._i64),
                         self._vector("loss", loss, rows, f32), self._vector("lse", lse, rows, f32),
                         self._stream(stream, x))
        return loss, lse

    def backward(self, x, w, target, lse, dloss=None, dlse=None, dx=None, dw=None, stream=None):
        """The gradients of `forward` that are asked for, from its lse and the
        gradients of loss (None: ones) and lse (None: zeros), float32 [rows]."""
        rows, f32 = x.shape[0], self._f32
        px, ldx = self._rows("x", x, rows, self.H)
        pw, ldw = self._rows("w", w, self.V, self.H)
        pdx, lddx = self._rows("dx", dx, rows, self.H)
        pdw, lddw = self._rows("dw", dw, self.V, self.H)
        mlp_loss_backward(self.h, rows, px, ldx, pw, ldw, self._vector("target", target, rows, self._i64),
                          self._vector("lse", lse, rows, f32), self._vector("dloss", dloss, rows, f32),
                          self._vector("dlse", dlse, rows, f32), pdx, lddx, pdw, lddw, self._stream(stream, x))
        return dx, dw


class MlpGradNorm(_Layer):
    """The norm of many gradients together, and the factor that clips it."""

    def __init__(self, dtype: str = "f16"):
        self._set_type(dtype)
        self._hold(mlp_grad_norm_create(DTYPES[dtype]))

    _destroy = staticmethod(mlp_grad_norm_destroy)

    def forward(self, grads, norm, scale=None, max_norm: float = math.inf, unscale: float = 1.0, stream=None):
        """norm = |unscale| sqrt(sum g^2) over the contiguous tensors `grads`; scale = unscale min(1, max_norm / norm),
        NaN if the norm is not finite (both float32 [1])."""
        from torch import Tensor
        n = len(grads)
        pointers = _pointers(self, "a gradient", grads, self.torch_dtype)
        sizes = _array(ctypes.c_int64, "q", map(Tensor.numel, grads), n)
        mlp_grad_norm_forward(self.h, n, sizes, pointers, float(unscale), float(max_norm),
                              self._vector("norm", norm, 1, self._f32), self._vector("scale", scale, 1, self._f32),
                              self._stream(stream, norm))
        return norm, scale


def _elements(layer, name, t, dtype):
    """Pointer of a contiguous tensor of any shape."""
    if t.dtype != dtype or t.get_device() != layer.device:
        raise ValueError(f"{name} must be a {dtype} tensor on the handle's device {layer.device}, got {t.dtype} on "
                         f"{t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, got strides {tuple(t.stride())}")
    return t.data_ptr()


def _pointers(layer, name, tensors, dtype):
    """A ctypes array of the pointers of contiguous tensors.  (A model has
    hundreds, a kernel over them takes tens of microseconds: each look at a
    tensor is one call of a C function for all, 0.04 us a tensor.)"""
    from torch import Tensor
    n = len(tensors)
    if ([t.dtype for t in tensors].count(dtype) != n or not all(map(Tensor.is_contiguous, tensors))
            or list(map(Tensor.get_device, tensors)).count(layer.device) != n):
        for t in tensors:
            _elements(layer, name, t, dtype)
    return _array(ctypes.c_void_p, "Q", map(Tensor.data_ptr, tensors), n)


def _array(kind, code, values, n):
    """A ctypes array of `values`."""
    values = array.array(code, values)
    return (kind * n).from_buffer(values) if n else (kind * 1)()


def _check_apart(lists):
    """Refuse contiguous tensors, given as (name, list) pairs, that share memory: a step writes all of them at once."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), name, i)
                   for name, ts in lists for i, t in enumerate(ts) if t.numel())
    for (_, end, a, i), (begin, _, b, k) in zip(spans, spans[1:]):
        if begin < end:
            raise ValueError(f"{a}[{i}] and {b}[{k}] share memory")


class MlpAdamW(_Layer):
    """AdamW over the contiguous tensors `params` of `dtype`, which it updates
    in place, with states of 32 or 8 bits, and with fp32 master weights if
    `master` is true.  States begin at zero, master weights at the parameters',
    and the step count at 0, unless they are given (a resumed run): `master`,
    `m` and `v` (one tensor per parameter, of its number of elements; float32,
    or of 8 bits float8_e4m3fn and float8_e5m2), `m_scale` and `v_scale`
    (float32, one per 256 elements) and `step` (int64 [1], counted on the
    device); none of these may share memory.  `decay`: weight decay, of all or
    of each.

    A step works on the memory that these tensors had here; a parameter that
    has got other memory since is refused.  The attributes `params`, `master`,
    `m`, `v`, `m_scale`, `v_scale` (lists; None where there are none) and `t`
    are what a checkpoint of the optimizer keeps."""

    def __init__(self, params, dtype: str = "f16", states: int = 32, beta1: float = 0.9, beta2: float = 0.999,
                 eps: float = 1e-8, decay=0.0, seed: int = 0, master=False, m=None, v=None, m_scale=None, v_scale=None,
                 step=None):
        import torch
        self._set_type(dtype)
        self.states = int(states)
        self._hold(mlp_adamw_create(DTYPES[dtype], states, beta1, beta2, eps, seed))
        self.params = list(params)
        n, f32 = len(self.params), torch.float32
        kinds = (f32, f32) if self.states == 32 else (torch.float8_e4m3fn, torch.float8_e5m2)
        pointers = _pointers(self, "a parameter", self.params, self.torch_dtype)
        sizes = [p.numel() for p in self.params]
        some = [p for p in list(pointers)[:n] if p]
        if len(set(some)) != len(some):
            raise ValueError("params has the same memory twice (a tied weight is one parameter)")
        blocks = [-(-k // BLOCK) for k in sizes]

        def given(name, tensors, dtype, sizes, make):
            tensors = list(tensors) if tensors is not None else [make(p, k) for p, k in zip(self.params, sizes)]
            if [t.numel() for t in tensors] != sizes:
                raise ValueError(f"{name} must have {n} tensors of {sizes} elements, got {[t.numel() for t in tensors]}")
            return tensors, _pointers(self, name, tensors, dtype)

        def zeros(kind):
            return lambda p, k: torch.zeros(p.shape, device=p.device, dtype=f32 if kind is f32 else torch.uint8).view(kind)

        self.master = self.m_scale = self.v_scale = masters = m_scales = v_scales = None
        if master is not None and master is not False:
            self.master, masters = given("master", None if master is True else master, f32, sizes, lambda p, k: p.detach().float())
        self.m, ms = given("m", m, kinds[0], sizes, zeros(kinds[0]))
        self.v, vs = given("v", v, kinds[1], sizes, zeros(kinds[1]))
        if self.states == 8:
            ones = lambda p, k: torch.ones(k, device=p.device)  # noqa: E731
            self.m_scale, m_scales = given("m_scale", m_scale, f32, blocks, ones)
            self.v_scale, v_scales = given("v_scale", v_scale, f32, blocks, ones)
        decays = [float(d) for d in decay] if hasattr(decay, "__len__") else [float(decay)] * n
        if len(decays) != n:
            raise ValueError(f"decay has {len(decays)} values, expected {n}")
        self.decay = decays
        at = lambda p, i: p[i] if p is not None else None  # noqa: E731
        self._table = (AdamwTensor * n)(*[
            AdamwTensor(sizes[i], pointers[i], at(masters, i), ms[i], vs[i], at(m_scales, i), at(v_scales, i), decays[i])
            for i in range(n)])
        self.t = torch.zeros(1, dtype=torch.int64, device=torch.device("cuda", self.device)) if step is None else step
        self._t = self._vector("step", self.t, 1, torch.int64)
        # (the memory behind the pointers stays while the optimizer does, whatever becomes of the tensors)
        lists = [(name, getattr(self, name)) for name in ("params", "master", "m", "v", "m_scale", "v_scale")] + [("step", [self.t])]
        lists = [(name, ts) for name, ts in lists if ts]
        _check_apart(lists)
        self._memory = [t.untyped_storage() for _, ts in lists for t in ts]
        self._params = list(pointers)[:n]
        self._shapes = [p.shape for p in self.params]
        # (what was made here is there for steps on any stream)
        torch.cuda.current_stream(self.device).synchronize()

    _destroy = staticmethod(mlp_adamw_destroy)

    def step(self, grads, lr: float, scale=None, lr_scale=None, stream=None):
        """One step with `grads`, one contiguous tensor per parameter, times `scale` (float32 [1] on the device); a scale
        that is not finite leaves the step out.  `lr_scale` (float32 [1] on the device) multiplies `lr`."""
        shapes = [g.shape for g in grads]
        if shapes != self._shapes:
            raise ValueError(f"grads has shapes {[tuple(s) for s in shapes]}, expected {[tuple(s) for s in self._shapes]}")
        if [p.data_ptr() or None for p in self.params] != self._params:
            raise ValueError("a parameter has got other memory since the optimizer was made")
        mlp_adamw_step(self.h, len(shapes), self._table, _pointers(self, "a gradient", grads, self.torch_dtype), float(lr),
                       self._vector("lr_scale", lr_scale, 1, self._f32), self._vector("scale", scale, 1, self._f32),
                       self._t, self._stream(stream, self.t))
