"""The attention half of a block: binding of the per-head norm and position
rotation of queries and keys, and of causal attention over packed sequences.

Like the rest of the binding, these functions only marshal arguments, the
launching ones through a small native module that checks every tensor's shape,
type, device and strides (csrc/marshal.cpp).  Tensors of heads are [rows, heads,
head_dim] with any row and head strides that are multiples of 8 (slices of a
fused projection, caches of either order).
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import numpy as np
import torch

from . import IPTTT_BF16, IPTTT_F32, _check, library

_DTYPES = {IPTTT_F32: torch.float32, IPTTT_BF16: torch.bfloat16}


class _CQKProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("table_rows", ctypes.c_int64), ("out_rows", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class _CAttnProblem(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("q_rows", ctypes.c_int64), ("k_rows", ctypes.c_int64),
                ("dtype", ctypes.c_int32)] + [(n, ctypes.POINTER(ctypes.c_int64))
                                              for n in ("q_start", "q_len", "k_start", "k_len")]


_bound = None
_calls = None


def _lib() -> ctypes.CDLL:
    """The library with this module's entry points declared."""
    global _bound
    if _bound is None:
        lib = library()
        vp, f32, i32, sz = ctypes.c_void_p, ctypes.c_float, ctypes.c_int, ctypes.c_size_t
        H = ctypes.c_char_p  # ipttt_heads, packed
        Q, A = ctypes.POINTER(_CQKProblem), ctypes.POINTER(_CAttnProblem)
        sigs = {
            "ipttt_qk_norm_rope": (i32, [Q, H, H, vp, vp, vp, vp, H, H, H, H, vp, vp]),
            "ipttt_qk_norm_rope_backward": (i32, [Q, H, H, vp, vp, vp, vp, H, H, H, H, vp, vp, vp, sz, vp]),
            "ipttt_qk_backward_workspace_bytes": (sz, [Q]),
            "ipttt_attn_validate": (i32, [A]),
            "ipttt_attn_plan_bytes": (sz, [A]),
            "ipttt_attn_plan": (i32, [A, vp, sz]),
            "ipttt_attn_workspace_bytes": (sz, [vp]),
            "ipttt_attn_backward_workspace_bytes": (sz, [vp]),
            "ipttt_attention": (i32, [vp, vp, f32, H, H, H, H, vp, vp, sz, vp]),
            "ipttt_attention_backward": (i32, [vp, vp, f32, H, H, H, H, vp, H, H, H, H, vp, sz, vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _bound = lib
    return _bound


def _native():
    """The marshalling module, bound to the library's launching entry points; it
    checks the tensors of a call and makes it."""
    global _calls
    if _calls is None:
        lib = _lib()
        try:
            from . import _marshal
        except ImportError as e:
            raise RuntimeError("the binding's _marshal.so is missing: build it with "
                               "`python -m test_weight_mlp_amd.build`") from e
        _marshal.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                        for n in ("ipttt_qk_norm_rope", "ipttt_qk_norm_rope_backward", "ipttt_attention",
                                  "ipttt_attention_backward")))
        _calls = _marshal
    return _calls


def _on(stream, q: torch.Tensor) -> int:
    """The given stream, or the current one.  Kernels are launched on the current
    device, so the tensors have to be there."""
    if not getattr(q, "is_cuda", False):  # refused with the other arguments
        return 0
    at, current = q.get_device(), torch._C._cuda_getDevice()
    if at != current:
        raise ValueError(f"q is on device {at}, the current device is {current}: call under torch.cuda.device({at})")
    # torch.cuda.current_stream() without its wrapper object
    return torch._C._cuda_getCurrentRawStream(at) if stream is None else stream.cuda_stream


# ------------------------------------------------------- norm and rotation

def rotation_table(positions: int, head_dim: int, theta: float, device="cuda") -> torch.Tensor:
    """[positions, head_dim] float32: cos, then sin, of position * theta^(-2 i /
    head_dim), computed in 64 bits (fp32 angles are off by 1e-2 at position 1e5)."""
    inv = float(theta) ** (-np.arange(0, head_dim, 2, dtype=np.float64) / head_dim)
    ang = np.arange(positions, dtype=np.float64)[:, None] * inv
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(device)


class QKProblem:
    """Sizes and dtype of one norm and rotation call (ipttt_qk_problem)."""

    def __init__(self, tokens: int, heads: int, kv_heads: int, head_dim: int, dtype: int = IPTTT_BF16,
                 eps: float = 1e-6, table_rows: int = 1, out_rows: Optional[int] = None):
        self.tokens, self.heads, self.kv_heads, self.head_dim = tokens, heads, kv_heads, head_dim
        self.dtype, self.eps, self.table_rows = dtype, eps, table_rows
        self.out_rows = tokens if out_rows is None else out_rows
        self._c = _CQKProblem(tokens, heads, kv_heads, head_dim, table_rows, self.out_rows, dtype, eps)
        self.ref = ctypes.byref(self._c)
        self.address = ctypes.addressof(self._c)

    @property
    def torch_dtype(self) -> torch.dtype:
        return _DTYPES[self.dtype]


def ipttt_qk_norm_rope(p: QKProblem, q, k, w_q, w_k, positions, table, q_out, k_out, v=None, v_out=None, rows=None,
                       stream=None):
    """Norms and rotates q and k into q_out and k_out; with ``rows`` the keys (and
    v, if given) go to those rows of k_out (and v_out).  q_out may be q."""
    if (v is None) != (v_out is None):
        raise ValueError("v and v_out go together")
    status = (_calls or _native()).qk(p.address, q, k, w_q, w_k, positions, table, q_out, k_out, v, v_out, rows,
                                      _on(stream, q))
    if status:
        _check(status, "ipttt_qk_norm_rope")


def ipttt_qk_backward_workspace_bytes(p: QKProblem) -> int:
    return int(_lib().ipttt_qk_backward_workspace_bytes(p.ref))


class QKGrads:
    """Device buffers of one backward of the norm and rotation."""

    def __init__(self, p: QKProblem, device="cuda"):
        dt, f32 = p.torch_dtype, torch.float32
        self.dq = torch.empty((p.tokens, p.heads, p.head_dim), dtype=dt, device=device)
        self.dk = torch.empty((p.tokens, p.kv_heads, p.head_dim), dtype=dt, device=device)
        self.dw_q = torch.empty(p.head_dim, dtype=f32, device=device)
        self.dw_k = torch.empty(p.head_dim, dtype=f32, device=device)
        self.ws = torch.empty(ipttt_qk_backward_workspace_bytes(p), dtype=torch.uint8, device=device)


def ipttt_qk_norm_rope_backward(p: QKProblem, q, k, w_q, w_k, positions, table, dq_out, dk_out, dq, dk, dw_q, dw_k, ws,
                                stream=None):
    status = (_calls or _native()).qk_backward(p.address, q, k, w_q, w_k, positions, table, dq_out, dk_out, dq, dk,
                                               dw_q, dw_k, ws, _on(stream, q))
    if status:
        _check(status, "ipttt_qk_norm_rope_backward")


# --------------------------------------------------------------- attention

class AttentionPlan:
    """Sequences of an attention call and the plan the library makes of them
    (ipttt_attn_problem, ipttt_attn_plan), on the host and the device; built
    once for a step and used by every layer.  It holds the lengths: a decoded token
    needs a new one (32 us for one sequence, 79 for 32, 374 for 256 of 8000 keys, with
    the copy to the device, which waits for it).  q_starts and k_starts default to
    sequences packed one after the other; scale defaults to head_dim^-1/2."""

    def __init__(self, heads: int, kv_heads: int, head_dim: int, q_lens: Sequence[int], k_lens: Sequence[int],
                 dtype: int = IPTTT_BF16, q_starts: Optional[Sequence[int]] = None,
                 k_starts: Optional[Sequence[int]] = None, q_rows: Optional[int] = None,
                 k_rows: Optional[int] = None, scale: Optional[float] = None, device="cuda"):
        def packed(starts, lens):
            s = np.concatenate([[0], np.cumsum(lens)[:-1]]) if starts is None else starts
            return np.ascontiguousarray(np.asarray(s, dtype=np.int64))

        ql, kl = (np.ascontiguousarray(np.asarray(x, dtype=np.int64)) for x in (q_lens, k_lens))
        arrays = [packed(q_starts, ql), ql, packed(k_starts, kl), kl]
        if any(x.ndim != 1 or x.size != ql.size for x in arrays):
            raise ValueError("q_lens, k_lens and their starts need one entry per sequence")
        ends = [int((s + n).max()) if n.size else 0 for s, n in (arrays[:2], arrays[2:])]
        self.heads, self.kv_heads, self.head_dim, self.dtype = heads, kv_heads, head_dim, dtype
        self.q_rows = ends[0] if q_rows is None else q_rows
        self.k_rows = ends[1] if k_rows is None else k_rows
        self.scale = 1.0 / math.sqrt(head_dim) if scale is None else float(scale)
        P = ctypes.POINTER(ctypes.c_int64)
        c = _CAttnProblem(ql.size, heads, kv_heads, head_dim, self.q_rows, self.k_rows, dtype,
                          *(P.from_buffer(ctypes.c_void_p(x.ctypes.data)) for x in arrays))
        lib, ref = _lib(), ctypes.byref(c)
        self._c, self._arrays = c, arrays  # the calls read the sizes
        self.address = ctypes.addressof(c)
        _check(lib.ipttt_attn_validate(ref), "ipttt_attn_validate")
        n = int(lib.ipttt_attn_plan_bytes(ref))
        self._host = np.empty((n + 7) // 8, dtype=np.int64)
        self.ref = self._host.ctypes.data
        _check(lib.ipttt_attn_plan(ref, self.ref, n), "ipttt_attn_plan")
        self.table = torch.from_numpy(self._host).to(device)
        self.workspace_bytes = int(lib.ipttt_attn_workspace_bytes(self.ref))
        self.backward_workspace_bytes = int(lib.ipttt_attn_backward_workspace_bytes(self.ref))

    @property
    def torch_dtype(self) -> torch.dtype:
        return _DTYPES[self.dtype]


class AttentionBuffers:
    """Outputs and workspace of the calls over one plan; with ``grads``, those of
    the backward too (one workspace serves both calls in turn)."""

    def __init__(self, plan: AttentionPlan, grads: bool = False, device="cuda"):
        dt, d = plan.torch_dtype, plan.head_dim
        q, k = (plan.q_rows, plan.heads, d), (plan.k_rows, plan.kv_heads, d)
        self.o = torch.empty(q, dtype=dt, device=device)
        self.lse = torch.empty(q[:2], dtype=torch.float32, device=device)
        need = max(plan.workspace_bytes, plan.backward_workspace_bytes if grads else 0)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        self.dq = torch.empty(q, dtype=dt, device=device) if grads else None
        self.dk = torch.empty(k, dtype=dt, device=device) if grads else None
        self.dv = torch.empty(k, dtype=dt, device=device) if grads else None


def ipttt_attention(plan: AttentionPlan, q, k, v, o, lse, ws=None, stream=None):
    status = (_calls or _native()).attention(plan.address, plan.ref, plan.scale, plan.table, q, k, v, o, lse, ws,
                                             _on(stream, q))
    if status:
        _check(status, "ipttt_attention")


def ipttt_attention_backward(plan: AttentionPlan, q, k, v, o, lse, dO, dq, dk, dv, ws, stream=None):
    status = (_calls or _native()).attention_backward(plan.address, plan.ref, plan.scale, plan.table, q, k, v, o, lse,
                                                      dO, dq, dk, dv, ws, _on(stream, q))
    if status:
        _check(status, "ipttt_attention_backward")
