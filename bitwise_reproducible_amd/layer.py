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
_NO_VIEW = (0, 0, 0, 0)
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


def _device(t, name: str) -> int:
    """The current device's index, on which t has to be."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on a ROCm device")
    device = torch.cuda.current_device()
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")
    return device


def _on(t, name: str, device: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on a ROCm device")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{device}")


def _current(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


def repro_rope_table(inv_freq, length: int, start: int = 0, cos=None, sin=None, stream=None):
    """(cos, sin) of (start + p) * inv_freq[i], float32 (length, len(inv_freq)); inv_freq float64."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_rope_table(inv_freq, length, start, cos, sin)
    device = _device(inv_freq, "inv_freq")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous 1-D float64 tensor")
    half = inv_freq.shape[0]
    length = int(length)
    if length < 0:
        raise ValueError("length must not be negative")
    tables = []
    for t, name in ((cos, "cos"), (sin, "sin")):
        if t is None:
            t = torch.empty((length, half), dtype=torch.float32, device=inv_freq.device)
        else:
            _on(t, name, device)
            if t.dtype != torch.float32 or tuple(t.shape) != (length, half) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor of shape {(length, half)}")
        tables.append(t)
    _base._check(_lib().repro_rope_table(inv_freq.data_ptr(), half, int(start), length, tables[0].data_ptr(),
                                         tables[1].data_ptr(), _current(device)), "repro_rope_table")
    return tables[0], tables[1]


def _view(t, name: str, device: int, dtype, shape):
    """(address, batch stride, token stride, head stride) of one side's tensor."""
    _on(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    b, s, h, d = t.stride()
    if d != 1:
        raise ValueError(f"{name} needs unit stride along its last dimension")
    return t.data_ptr(), b, s, h


def _common(q, k, cos, sin, positions, q_gain, k_gain):
    """What both passes check alike: (device, the packed fields up to the gains)."""
    device = _device(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be (batch, seq, heads, dim)")
    if q.dtype not in _TYPES:
        raise TypeError("q must be float32 or bfloat16")
    _on(k, "k", device)
    if k.dim() != 4 or k.shape[0] != q.shape[0] or k.shape[1] != q.shape[1] or k.shape[3] != q.shape[3]:
        raise ValueError("k must be (batch, seq, heads, dim) with q's batch, seq and dim")
    batch, seq, q_heads, dim = q.shape
    for t, name in ((cos, "cos"), (sin, "sin")):
        _on(t, name, device)
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be {torch.float32}, not {t.dtype}")
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise ValueError("cos and sin must be (positions, rotary / 2) and of one shape")
    rows, half = cos.shape
    stride = cos.stride(0) if rows > 1 else half
    if half > 1 and (cos.stride(1) != 1 or sin.stride(1) != 1) or rows > 1 and sin.stride(0) != stride:
        raise ValueError("cos and sin need unit stride along their last dimension and one row stride")
    at, size, strides = 0, 0, (0, 0)
    if positions is not None:
        _on(positions, "positions", device)
        if positions.dtype not in (torch.int32, torch.int64):
            raise TypeError("positions must be int32 or int64")
        if positions.dim() == 1 and positions.shape[0] == seq:
            strides = (0, positions.stride(0))
        elif positions.dim() == 2 and positions.shape[0] == batch and positions.shape[1] == seq:
            strides = positions.stride()
        else:
            raise ValueError("positions must be (batch, seq) or (seq,)")
        # No element: any address will do, since none is read.
        at, size = positions.data_ptr() or 16, positions.element_size()
    gain_type, gains = None, [0, 0]
    for i, (t, name) in enumerate(((q_gain, "q_gain"), (k_gain, "k_gain"))):
        if t is None:
            continue
        _on(t, name, device)
        if t.dtype not in _TYPES or gain_type not in (None, t.dtype):
            raise TypeError("the gains must be float32 or bfloat16, and of one type")
        if t.dim() != 1 or t.shape[0] != dim or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of {dim} elements")
        gain_type = t.dtype
        gains[i] = t.data_ptr()
    fields = (cos.data_ptr(), sin.data_ptr(), rows, stride, at, *strides, *gains)
    head = (batch, seq, q_heads, k.shape[2], dim, 2 * half, _TYPES[q.dtype], _TYPES.get(gain_type, 0))
    return device, head, size, fields


def repro_qk_norm_rope(q, k, cos, sin, positions=None, q_gain=None, k_gain=None, eps: float = 1e-6,
                       interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Every query and key head normalised, scaled by its gain and rotated by its position (see repro.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved, q_out, k_out)
    device, head, size, fields = _common(q, k, cos, sin, positions, q_gain, k_gain)
    dtype = q.dtype
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=dtype, device=q.device)
    args = _QK.pack(*head, 1 if interleaved else 0, size, *fields,
                    *_view(q, "q", device, dtype, q.shape), *_view(k, "k", device, dtype, k.shape),
                    *_view(q_out, "q_out", device, dtype, q.shape), *_view(k_out, "k_out", device, dtype, k.shape),
                    *_NO_VIEW, *_NO_VIEW, 0, 0, eps, 0)
    _base._check(_lib().repro_qk_norm_rope(args, _current(device)), "repro_qk_norm_rope")
    return q_out, k_out


def repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions=None, q_gain=None, k_gain=None,
                                eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, dq_gain=None,
                                dk_gain=None, workspace=None, stream=None):
    """Gradients of repro_qk_norm_rope at (q, k) for the outputs' gradients dq_out, dk_out: (dq, dk, dq_gain,
    dk_gain), the gains' in float32 (None where there is no gain)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions, q_gain, k_gain, eps,
                                               interleaved, dq, dk, dq_gain, dk_gain, workspace)
    device, head, size, fields = _common(q, k, cos, sin, positions, q_gain, k_gain)
    dtype, where = q.dtype, q.device
    if dq is None:
        dq = torch.empty(q.shape, dtype=dtype, device=where)
    if dk is None:
        dk = torch.empty(k.shape, dtype=dtype, device=where)
    grads = []
    for gain, t, name in ((q_gain, dq_gain, "dq_gain"), (k_gain, dk_gain, "dk_gain")):
        if gain is None:
            if t is not None:
                raise ValueError(f"{name} without its gain")
        elif t is None:
            t = torch.empty(gain.shape, dtype=torch.float32, device=where)
        else:
            _on(t, name, device)
            if t.dtype != torch.float32 or t.shape != gain.shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor of {gain.shape[0]} elements")
        grads.append(t)
    args = _QK.pack(*head, 1 if interleaved else 0, size, *fields,
                    *_view(q, "q", device, dtype, q.shape), *_view(k, "k", device, dtype, k.shape),
                    *_view(dq, "dq", device, dtype, q.shape), *_view(dk, "dk", device, dtype, k.shape),
                    *_view(dq_out, "dq_out", device, dtype, q.shape),
                    *_view(dk_out, "dk_out", device, dtype, k.shape),
                    *(0 if t is None else t.data_ptr() for t in grads), eps, 0)
    lib = _lib()
    at, room = 0, 0
    if q_gain is not None or k_gain is not None:
        if workspace is None:
            need = lib.repro_qk_workspace_bytes(args)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=where)
        else:
            _base._on_device(workspace, "workspace", torch.uint8)
        if workspace is not None:
            at, room = workspace.data_ptr(), workspace.numel()
    _base._check(lib.repro_qk_norm_rope_backward(args, at, room, _current(device)), "repro_qk_norm_rope_backward")
    return dq, dk, grads[0], grads[1]


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
            out = torch.empty(3, dtype=torch.float32, device=self._plan.device)
        else:
            _base._on_device(out, "out", torch.float32, 12)
        current = _current(device)
        if current != self._stream:  # the plan's memory is the other stream's
            self._plan.record_stream(torch.cuda.current_stream())
        _base._check(getattr(_lib(), what)(self._head, self._plan.data_ptr(), *args, out.data_ptr(), current), what)
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
