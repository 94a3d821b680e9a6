"""Operators around one attention layer and one optimizer step (binding).

Argument marshalling as in the package's other entry points (OPEN-1B paper,
section 3.1: rotary positions and a norm of every query and key head; section
3.2 "Optimizer": the global-norm clip).  All of these are attributes of the
package too:

    repro_rope_table(inv_freq, length, start=0, cos=None, sin=None) -> (cos, sin)
    repro_qk_norm_rope(q, k, cos, sin, positions=None, q_gain=None, k_gain=None, eps=1e-6,
                       interleaved=False, q_out=None, k_out=None) -> (q_out, k_out)
    repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions=None, q_gain=None, k_gain=None,
                                eps=1e-6, interleaved=False, dq=None, dk=None, dq_gain=None, dk_gain=None,
                                workspace=None) -> (dq, dk, dq_gain, dk_gain)
    GradList(grads, outs=None)
    repro_grad_list_norm(list, out=None) -> device tensor [norm, S, 1]
    repro_clip_grad_list(list, max_norm, out=None) -> device tensor [norm, S, coef]

Queries and keys are (batch, seq, heads, dim) tensors of float32 or bfloat16
with any strides of the first three dimensions (so parts of one projection's
output, and heads before tokens, are taken where they lie).  `stream` orders
everything a call does, its own allocations too; without it that is the
current stream.
"""
from __future__ import annotations

import ctypes
import struct

import torch

import bitwise_reproducible_amd as _base

# repro_qk_args (include/repro.h).
_QK = struct.Struct("@qq8iPPqqPqqPP" + "Pqqq" * 6 + "PPfi")
_TYPES = {torch.float32: 0, torch.bfloat16: 1}
_bound = None


def _lib():
    """The library, with these entry points' argument types set."""
    global _bound
    if _bound is None:
        lib = _base.library()
        i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
        lib.repro_rope_table.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        lib.repro_qk_norm_rope.argtypes = [ctypes.c_char_p, vp]
        lib.repro_qk_workspace_bytes.argtypes = [ctypes.c_char_p]
        lib.repro_qk_workspace_bytes.restype = i64
        lib.repro_qk_norm_rope_backward.argtypes = [ctypes.c_char_p, vp, i64, vp]
        lib.repro_grad_list_bytes.argtypes = [vp, vp, i64]
        lib.repro_grad_list_bytes.restype = i64
        lib.repro_grad_list_plan.argtypes = [vp, vp, vp, vp, i64, vp, i64]
        lib.repro_grad_list_norm.argtypes = [vp, vp, vp, vp]
        lib.repro_clip_grad_list.argtypes = [vp, vp, f32, vp, vp]
        for name in ("repro_rope_table", "repro_qk_norm_rope", "repro_qk_norm_rope_backward", "repro_grad_list_plan",
                     "repro_grad_list_norm", "repro_clip_grad_list"):
            getattr(lib, name).restype = ctypes.c_int
        _bound = lib
    return _bound


_Tensor = torch.Tensor
_F32 = torch.float32
_current = torch._C._cuda_getCurrentRawStream  # a device's current stream, as the library takes it


def _device(t, name: str) -> int:
    """The current device's index, on which t has to be."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on a ROCm device")
    device = torch.cuda.current_device()
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    return device


def _on(t, name: str, device: int):
    if not isinstance(t, _Tensor) or t.get_device() != device:
        _device(t, name)


def repro_rope_table(inv_freq, length: int, start: int = 0, cos=None, sin=None, stream=None):
    """(cos, sin) of (start + p) * inv_freq[i], float32 (length, len(inv_freq)); inv_freq float64."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_rope_table(inv_freq, length, start, cos, sin)
    device = _device(inv_freq, "inv_freq")
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous 1-D float64 tensor")
    half = inv_freq.shape[0]
    length = int(length)
    if length < 0:
        raise ValueError("length must not be negative")
    if cos is None:
        cos = torch.empty((length, half), dtype=_F32, device=inv_freq.device)
    else:
        _table_out(cos, "cos", device, length, half)
    if sin is None:
        sin = torch.empty_like(cos)
    else:
        _table_out(sin, "sin", device, length, half)
    status = _lib().repro_rope_table(inv_freq.data_ptr(), half, int(start), length, cos.data_ptr(), sin.data_ptr(),
                                     _current(device))
    if status:
        raise _base.ReproError(status, "repro_rope_table")
    return cos, sin


def _table_out(t, name: str, device: int, length: int, half: int):
    _on(t, name, device)
    if t.dtype is not _F32 or t.shape != (length, half) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(length, half)}")


def _view(t, name: str, device: int, dtype, shape):
    """(address, batch stride, token stride, head stride) of one side's tensor."""
    if not isinstance(t, _Tensor) or t.get_device() != device:
        _device(t, name)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    b, s, h, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} needs unit stride along its last dimension")
    return t.data_ptr(), b, s, h


def _common(q, k, cos, sin, positions, q_gain, k_gain, interleaved):
    """What both passes check alike: (device, type, q's shape, k's shape, the packed fields up to the views)."""
    device = _device(q, "q")
    dtype = q.dtype
    kind = _TYPES.get(dtype)
    if kind is None:
        raise TypeError("q must be float32 or bfloat16")
    _on(k, "k", device)
    q_shape, k_shape = q.shape, k.shape
    if len(q_shape) != 4:
        raise ValueError("q must be (batch, seq, heads, dim)")
    batch, seq, q_heads, dim = q_shape
    if len(k_shape) != 4 or k_shape[0] != batch or k_shape[1] != seq or k_shape[3] != dim:
        raise ValueError("k must be (batch, seq, heads, dim) with q's batch, seq and dim")
    _on(cos, "cos", device)
    _on(sin, "sin", device)
    if cos.dtype is not _F32 or sin.dtype is not _F32:
        raise TypeError(f"cos and sin must be {_F32}")
    table, strides = cos.shape, cos.stride()
    if len(table) != 2 or sin.shape != table:
        raise ValueError("cos and sin must be (positions, rotary / 2) and of one shape")
    rows, half = table
    stride, unit = strides
    if rows > 1 and half > 1:
        plain = unit == 1 and sin.stride() == strides
    else:  # a dimension of one element has any stride
        plain = (half <= 1 or unit == 1 and sin.stride(1) == 1) and (rows <= 1 or sin.stride(0) == stride)
        stride = stride if rows > 1 else half
    if not plain:
        raise ValueError("cos and sin need unit stride along their last dimension and one row stride")
    at, size, by_batch, by_seq = 0, 0, 0, 0
    if positions is not None:
        _on(positions, "positions", device)
        size = 4 if positions.dtype is torch.int32 else 8
        if size == 8 and positions.dtype is not torch.int64:
            raise TypeError("positions must be int32 or int64")
        where = positions.shape
        if where == (batch, seq):
            by_batch, by_seq = positions.stride()
        elif where == (seq,):
            by_seq = positions.stride(0)
        else:
            raise ValueError("positions must be (batch, seq) or (seq,)")
        at = positions.data_ptr() or 16  # without elements any address will do, since none is read
    q_at, k_at, gain_kind = 0, 0, 0
    if q_gain is not None or k_gain is not None:
        q_at = _gain(q_gain, "q_gain", device, dim)
        k_at = _gain(k_gain, "k_gain", device, dim)
        gain = q_gain if q_gain is not None else k_gain
        if k_gain is not None and k_gain.dtype is not gain.dtype:
            raise TypeError("the gains must be of one type")
        gain_kind = _TYPES[gain.dtype]
    return device, dtype, q_shape, k_shape, (batch, seq, q_heads, k_shape[2], dim, 2 * half, kind, gain_kind,
                                             1 if interleaved else 0, size, cos.data_ptr(), sin.data_ptr(), rows,
                                             stride, at, by_batch, by_seq, q_at, k_at)


def _gain(t, name: str, device: int, dim: int) -> int:
    if t is None:
        return 0
    _on(t, name, device)
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if t.shape != (dim,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {dim} elements")
    return t.data_ptr()


def repro_qk_norm_rope(q, k, cos, sin, positions=None, q_gain=None, k_gain=None, eps: float = 1e-6,
                       interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Every query and key head normalised, scaled by its gain and rotated by its position (see repro.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved, q_out, k_out)
    device, dtype, q_shape, k_shape, fields = _common(q, k, cos, sin, positions, q_gain, k_gain, interleaved)
    if q_out is None:
        q_out = torch.empty(q_shape, dtype=dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k_shape, dtype=dtype, device=q.device)
    args = _QK.pack(*fields, *_view(q, "q", device, dtype, q_shape), *_view(k, "k", device, dtype, k_shape),
                    *_view(q_out, "q_out", device, dtype, q_shape), *_view(k_out, "k_out", device, dtype, k_shape),
                    0, 0, 0, 0, 0, 0, 0, 0, 0, 0, eps, 0)
    status = (_bound or _lib()).repro_qk_norm_rope(args, _current(device))
    if status:
        raise _base.ReproError(status, "repro_qk_norm_rope")
    return q_out, k_out


def _gain_grad(gain, t, name: str, device: int):
    """The tensor for a gain's gradient; None without a gain."""
    if gain is None:
        if t is not None:
            raise ValueError(f"{name} without its gain")
        return None
    if t is None:
        return torch.empty(gain.shape, dtype=_F32, device=gain.device)
    _on(t, name, device)
    if t.dtype is not _F32 or t.shape != gain.shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {gain.shape[0]} elements")
    return t


def repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions=None, q_gain=None, k_gain=None,
                                eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, dq_gain=None,
                                dk_gain=None, workspace=None, stream=None):
    """Gradients of repro_qk_norm_rope at (q, k) for the outputs' gradients dq_out, dk_out: (dq, dk, dq_gain,
    dk_gain), the gains' in float32 (None where there is no gain)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions, q_gain, k_gain, eps,
                                               interleaved, dq, dk, dq_gain, dk_gain, workspace)
    device, dtype, q_shape, k_shape, fields = _common(q, k, cos, sin, positions, q_gain, k_gain, interleaved)
    if dq is None:
        dq = torch.empty(q_shape, dtype=dtype, device=q.device)
    if dk is None:
        dk = torch.empty(k_shape, dtype=dtype, device=q.device)
    dq_gain = _gain_grad(q_gain, dq_gain, "dq_gain", device)
    dk_gain = _gain_grad(k_gain, dk_gain, "dk_gain", device)
    args = _QK.pack(*fields, *_view(q, "q", device, dtype, q_shape), *_view(k, "k", device, dtype, k_shape),
                    *_view(dq, "dq", device, dtype, q_shape), *_view(dk, "dk", device, dtype, k_shape),
                    *_view(dq_out, "dq_out", device, dtype, q_shape),
                    *_view(dk_out, "dk_out", device, dtype, k_shape),
                    0 if dq_gain is None else dq_gain.data_ptr(), 0 if dk_gain is None else dk_gain.data_ptr(), eps, 0)
    lib = _bound or _lib()
    at, room = 0, 0
    if dq_gain is not None or dk_gain is not None:
        if workspace is None:
            need = lib.repro_qk_workspace_bytes(args)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _base._on_device(workspace, "workspace", torch.uint8)
        if workspace is not None:
            at, room = workspace.data_ptr(), workspace.numel()
    status = lib.repro_qk_norm_rope_backward(args, at, room, _current(device))
    if status:
        raise _base.ReproError(status, "repro_qk_norm_rope_backward")
    return dq, dk, dq_gain, dk_gain


class GradList:
    """A list of gradient tensors (contiguous float32 or bfloat16, any sizes and types mixed) laid out once for
    repro_grad_list_norm and repro_clip_grad_list.

    outs: tensors for the clipped gradients, of the same types and sizes; an out may be its own gradient, and
    without outs all are (in place).  The list stands for the memory these tensors have now: it keeps the tensors,
    and a new list is needed when a gradient moves.  Calls on one list share its workspace, so they must be ordered.
    """

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("outs must have one tensor for each gradient")
        device = None
        for name, ts in (("grads", self.grads), ("outs", self.outs)):
            for i, t in enumerate(ts):
                what = f"{name}[{i}]"
                device = _device(t, what) if device is None else device
                _on(t, what, device)
                if t.dtype not in _TYPES or t.dtype != self.grads[i].dtype:
                    raise TypeError(f"{what} must be float32 or bfloat16, an out of its gradient's type")
                if not t.is_contiguous() or t.numel() != self.grads[i].numel():
                    raise ValueError(f"{what} must be contiguous, an out of its gradient's size")
        self.device = torch.cuda.current_device() if device is None else device
        n = len(self.grads)
        ptrs = [(ctypes.c_void_p * n)(*[t.data_ptr() for t in ts]) for ts in (self.grads, self.outs)]
        sizes = (ctypes.c_int64 * n)(*[t.numel() for t in self.grads])
        types = (ctypes.c_int32 * n)(*[_TYPES[t.dtype] for t in self.grads])
        lib = _lib()
        nbytes = lib.repro_grad_list_bytes(sizes, types, n)
        if nbytes < 0:
            raise _base.ReproError(int(nbytes), "repro_grad_list_bytes")
        host = torch.empty(nbytes, dtype=torch.uint8)
        _base._check(lib.repro_grad_list_plan(ptrs[0], ptrs[1], sizes, types, n, host.data_ptr(), nbytes),
                     "repro_grad_list_plan")
        self._plan = host.to(f"cuda:{self.device}")  # returns after the copy, so any stream may use it
        self._where = self._plan.device
        self._at = self._plan.data_ptr()
        self._head = bytes(host[:64].numpy())
        self._stream = _current(self.device)

    def __len__(self):
        return len(self.grads)

    def _call(self, what: str, out, stream, *args):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._call(what, out, None, *args)
        device = torch.cuda.current_device()
        if device != self.device:
            raise ValueError(f"the list is on cuda:{self.device}, but the current device is cuda:{device}")
        if out is None:
            out = torch.empty(3, dtype=_F32, device=self._where)
        else:
            _base._on_device(out, "out", _F32, 12)
        current = _current(device)
        if current != self._stream:  # the plan's memory is the other stream's
            self._plan.record_stream(torch.cuda.current_stream())
        status = getattr(_bound or _lib(), what)(self._head, self._at, *args, out.data_ptr(), current)
        if status:
            raise _base.ReproError(status, what)
        return out


def _grad_list(t):
    if not isinstance(t, GradList):
        raise TypeError("the list must be a GradList of tensors on a ROCm device")
    return t


def repro_grad_list_norm(grads, out=None, stream=None):
    """Device tensor [norm, S, 1]: the global l2 norm of a GradList and its square sum."""
    return _grad_list(grads)._call("repro_grad_list_norm", out, stream)


def repro_clip_grad_list(grads, max_norm: float, out=None, stream=None):
    """Clips a GradList to a global l2 norm of max_norm into its outs; device tensor [norm, S, coef]."""
    return _grad_list(grads)._call("repro_clip_grad_list", out, stream, float(max_norm))


# The package's __all__ lists the calls of its own file; these are attributes of the package as well.
__all__ = ["GradList", "repro_rope_table", "repro_qk_norm_rope", "repro_qk_norm_rope_backward",
           "repro_grad_list_norm", "repro_clip_grad_list"]
