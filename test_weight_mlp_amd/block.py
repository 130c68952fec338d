"""The rest of a block: binding of the norm in front of each half and of the
projections of the attention half with their epilogue.

Like the attention half's binding, the calls only marshal arguments, through the
native module that checks every tensor's shape, type, device and strides
(csrc/marshal.cpp).  Row tensors are [rows, columns] with any row stride that is
a multiple of 8 (columns of a wider tensor).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import IPTTT_BF16, IPTTT_F32, _check, library

IPTTT_NORM_RMS = 0
IPTTT_NORM_LAYER = 1
IPTTT_ACT_NONE = 0
IPTTT_ACT_SILU = 1
IPTTT_ACT_GELU = 2

_DTYPES = {IPTTT_F32: torch.float32, IPTTT_BF16: torch.bfloat16}


class _CNormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("eps", ctypes.c_float)]


class _CLinearProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


_bound = None
_calls = None


def _lib() -> ctypes.CDLL:
    """The library with this module's entry points declared."""
    global _bound
    if _bound is None:
        lib = library()
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        R = ctypes.c_char_p  # ipttt_rows, packed
        N, L = ctypes.POINTER(_CNormProblem), ctypes.POINTER(_CLinearProblem)
        sigs = {
            "ipttt_norm": (i32, [N, R, vp, vp, R, vp]),
            "ipttt_norm_backward_workspace_bytes": (sz, [N]),
            "ipttt_norm_backward": (i32, [N, R, vp, R, R, R, vp, vp, vp, sz, vp]),
            "ipttt_linear_workspace_bytes": (sz, [L]),
            "ipttt_linear": (i32, [L, R, vp, vp, R, R, R, vp, sz, vp]),
            "ipttt_linear_backward_workspace_bytes": (sz, [L]),
            "ipttt_linear_backward": (i32, [L, R, vp, R, R, R, vp, vp, vp, sz, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _bound = lib
    return _bound


def _native():
    """The marshalling module, bound to the library's launching entry points."""
    global _calls
    if _calls is None:
        lib = _lib()
        try:
            from . import _marshal
        except ImportError as e:
            raise RuntimeError("the binding's _marshal.so is missing: build it with "
                               "`python -m test_weight_mlp_amd.build`") from e
        _marshal.bind_block(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                              for n in ("ipttt_norm", "ipttt_norm_backward", "ipttt_linear",
                                        "ipttt_linear_backward")))
        _calls = _marshal
    return _calls


def _on(stream, x: torch.Tensor) -> int:
    """The given stream, or the current one.  Kernels are launched on the current
    device, so the tensors have to be there."""
    if not getattr(x, "is_cuda", False):  # refused with the other arguments
        return 0
    at, current = x.get_device(), torch._C._cuda_getDevice()
    if at != current:
        raise ValueError(f"x is on device {at}, the current device is {current}: call under torch.cuda.device({at})")
    return torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream


def _workspace(need: int, device):
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


# -------------------------------------------------------------------- norm

class NormProblem:
    """Sizes, dtype and kind of one norm call (ipttt_norm_problem)."""

    def __init__(self, rows: int, dim: int, dtype: int = IPTTT_BF16, kind: int = IPTTT_NORM_RMS, eps: float = 1e-6):
        self.rows, self.dim, self.dtype, self.kind, self.eps = rows, dim, dtype, kind, eps
        self._c = _CNormProblem(rows, dim, dtype, kind, eps)
        self.ref = ctypes.byref(self._c)
        self.address = ctypes.addressof(self._c)

    @property
    def torch_dtype(self) -> torch.dtype:
        return _DTYPES[self.dtype]


def ipttt_norm(p: NormProblem, x, w, b, y, stream=None):
    """The norm of x's rows times w plus b (either None) into y, which may be x."""
    status = (_calls or _native()).norm(p.address, x, w, b, y, _on(stream, x))
    if status:
        _check(status, "ipttt_norm")


def ipttt_norm_backward_workspace_bytes(p: NormProblem) -> int:
    return int(_lib().ipttt_norm_backward_workspace_bytes(p.ref))


class NormGrads:
    """Device buffers of one backward of the norm."""

    def __init__(self, p: NormProblem, device="cuda"):
        self.dx = torch.empty((p.rows, p.dim), dtype=p.torch_dtype, device=device)
        self.dw, self.db = (torch.empty(p.dim, dtype=torch.float32, device=device) for _ in "wb")
        self.ws = _workspace(ipttt_norm_backward_workspace_bytes(p), device)


def ipttt_norm_backward(p: NormProblem, x, w, dy, dx, dw, db, ws, dres=None, stream=None):
    """dx (plus dres), dw and db (either None) from the cotangent dy; dx may be x, dy or dres."""
    status = (_calls or _native()).norm_backward(p.address, x, w, dy, dres, dx, dw, db, ws, _on(stream, x))
    if status:
        _check(status, "ipttt_norm_backward")


# ------------------------------------------------------------- projections

class LinearProblem:
    """Sizes, dtype and activation of one projection (ipttt_linear_problem);
    grad_dtype is the type of dW: dtype (the default) or IPTTT_F32."""

    def __init__(self, rows: int, in_dim: int, out_dim: int, dtype: int = IPTTT_BF16, act: int = IPTTT_ACT_NONE,
                 grad_dtype: Optional[int] = None):
        self.rows, self.in_dim, self.out_dim, self.dtype, self.act = rows, in_dim, out_dim, dtype, act
        self.grad_dtype = dtype if grad_dtype is None else grad_dtype
        self._c = _CLinearProblem(rows, in_dim, out_dim, dtype, act, self.grad_dtype)
        self.ref = ctypes.byref(self._c)
        self.address = ctypes.addressof(self._c)

    @property
    def torch_dtype(self) -> torch.dtype:
        return _DTYPES[self.dtype]


def ipttt_linear_workspace_bytes(p: LinearProblem) -> int:
    return int(_lib().ipttt_linear_workspace_bytes(p.ref))


def linear_workspace(p: LinearProblem, device="cuda") -> Optional[torch.Tensor]:
    """A workspace for ipttt_linear; None where it needs none."""
    return _workspace(ipttt_linear_workspace_bytes(p), device)


def ipttt_linear(p: LinearProblem, x, W, y, b=None, res=None, pre=None, ws=None, stream=None):
    """y = act(x W^T + b) + res, y and res may be one tensor; pre receives x W^T + b."""
    status = (_calls or _native()).linear(p.address, x, W, b, res, y, pre, ws, _on(stream, x))
    if status:
        _check(status, "ipttt_linear")


def ipttt_linear_backward_workspace_bytes(p: LinearProblem) -> int:
    return int(_lib().ipttt_linear_backward_workspace_bytes(p.ref))


class LinearGrads:
    """Device buffers of one backward of a projection."""

    def __init__(self, p: LinearProblem, device="cuda"):
        self.dx = torch.empty((p.rows, p.in_dim), dtype=p.torch_dtype, device=device)
        self.dW = torch.empty((p.out_dim, p.in_dim), dtype=_DTYPES[p.grad_dtype], device=device)
        self.db = torch.empty(p.out_dim, dtype=torch.float32, device=device)
        self.ws = _workspace(ipttt_linear_backward_workspace_bytes(p), device)


def ipttt_linear_backward(p: LinearProblem, x, W, dy, dx, dW, db, ws, pre=None, stream=None):
    """dx, dW and db (each None: not wanted) from the cotangent dy; pre as the
    forward kept it, where the problem has an activation."""
    status = (_calls or _native()).linear_backward(p.address, x, W, pre, dy, dx, dW, db, ws, _on(stream, x))
    if status:
        _check(status, "ipttt_linear_backward")
