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
output, and heads before tokens, are taken where they lie).  No output may
share memory with another tensor of its call, but for a result over its side's
own input.  `stream` orders everything a call does, its own allocations too;
without it that is the current stream.  As with the package's other calls,
autograd records none of them: the backward pass is a call of its own.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

import bitwise_reproducible_amd as _base

EXTENSION_PATH = os.path.join(_base._HERE, "_layer.so")
_current = torch._C._cuda_getCurrentRawStream  # a device's current stream, as the library takes it
_bound = None
_calls = None


def _lib():
    """The library, with these entry points' argument types set."""
    global _bound
    if _bound is None:
        lib = _base.library()
        i32, i64, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
        lib.repro_rope_table.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        lib.repro_qk_norm_rope.argtypes = [vp, vp]
        lib.repro_qk_workspace_bytes.argtypes = [vp]
        lib.repro_qk_workspace_bytes.restype = i64
        lib.repro_qk_norm_rope_backward.argtypes = [vp, vp, i64, vp]
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


def _load():
    """The extension that checks tensors and calls the library (csrc/layer_binding.cpp)."""
    global _calls
    if _calls is None:
        if not os.path.exists(EXTENSION_PATH):
            raise RuntimeError(f"{EXTENSION_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; "
                               f"g.build()'`; there is no fallback path")
        lib = _lib()
        spec = importlib.util.spec_from_file_location("_layer", EXTENSION_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        entry = [ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "repro_rope_table", "repro_qk_norm_rope", "repro_qk_workspace_bytes", "repro_qk_norm_rope_backward",
            "repro_grad_list_bytes", "repro_grad_list_plan", "repro_grad_list_norm", "repro_clip_grad_list")]
        module.bind(*entry, _current)
        _calls = module
    return _calls


def _done(result, what: str):
    """The call's tensors; a status in their place is an error."""
    if result.__class__ is int:
        raise _base.ReproError(result, what)
    return result


def repro_rope_table(inv_freq, length: int, start: int = 0, cos=None, sin=None, stream=None):
    """(cos, sin) of (start + p) * inv_freq[i], float32 (length, len(inv_freq)); inv_freq float64.  Rounded once from
    values within 7e-15 of the exact ones."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_rope_table(inv_freq, length, start, cos, sin)
    return _done((_calls or _load()).rope_table(inv_freq, length, start, cos, sin), "repro_rope_table")


def repro_qk_norm_rope(q, k, cos, sin, positions=None, q_gain=None, k_gain=None, eps: float = 1e-6,
                       interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Every query and key head normalised, scaled by its gain and rotated by its position (see repro.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved, q_out, k_out)
    return _done((_calls or _load()).qk(q, k, cos, sin, positions, q_gain, k_gain, eps, interleaved, q_out, k_out),
                 "repro_qk_norm_rope")


def repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions=None, q_gain=None, k_gain=None,
                                eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, dq_gain=None,
                                dk_gain=None, workspace=None, stream=None):
    """Gradients of repro_qk_norm_rope at (q, k) for the outputs' gradients dq_out, dk_out: (dq, dk, dq_gain,
    dk_gain), the gains' in float32 (None where there is no gain)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_qk_norm_rope_backward(q, k, dq_out, dk_out, cos, sin, positions, q_gain, k_gain, eps,
                                               interleaved, dq, dk, dq_gain, dk_gain, workspace)
    return _done((_calls or _load()).qk_backward(q, k, dq_out, dk_out, cos, sin, positions, q_gain, k_gain, eps,
                                                 interleaved, dq, dk, dq_gain, dk_gain, workspace),
                 "repro_qk_norm_rope_backward")


class GradList:
    """A list of gradient tensors (contiguous float32 or bfloat16, any sizes and types mixed) laid out once for
    repro_grad_list_norm and repro_clip_grad_list.

    outs: tensors for the clipped gradients, of the same types and sizes; an out may be its own gradient, and
    without outs all are (in place).  The list keeps the tensors and stands for the memory they have now: a call
    refuses a list of which a tensor has moved.  It cannot see that a parameter was given another gradient tensor, as
    torch's zero_grad() does: it would go on clipping the old ones.  Keep gradients in buffers that stay
    (zero_grad(set_to_none=False), or views of one flat buffer), or make a new list.  Calls on one list share its
    workspace, so they must be ordered.
    """

    def __init__(self, grads, outs=None):
        self.grads = tuple(grads)
        self.outs = self.grads if outs is None else tuple(outs)
        self.device, host, self._held = _done((_calls or _load()).list_plan(self.grads, self.outs),
                                              "repro_grad_list_plan")
        self._plan = host.to(f"cuda:{self.device}")  # returns after the copy, so any stream may use it
        self._head = bytes(host[:64].numpy())
        self._stream = _current(self.device)

    def __len__(self):
        return len(self.grads)

    def _call(self, what: str, max_norm, out, stream):
        if stream is not None:
            with torch.cuda.stream(stream):
                return self._call(what, max_norm, out, None)
        if _current(self.device) != self._stream:  # the plan's memory is the other stream's
            self._plan.record_stream(torch.cuda.current_stream(self.device))
        return _done((_calls or _load()).grad_list(self._head, self._plan, max_norm, out, self.grads, self.outs,
                                                     self._held), what)


def _grad_list(t):
    if not isinstance(t, GradList):
        raise TypeError("the list must be a GradList of tensors on a ROCm device")
    return t


def repro_grad_list_norm(grads, out=None, stream=None):
    """Device tensor [norm, S, 1]: the global l2 norm of a GradList and its square sum.  out may share no memory with
    the list's tensors."""
    return _grad_list(grads)._call("repro_grad_list_norm", None, out, stream)


def repro_clip_grad_list(grads, max_norm: float, out=None, stream=None):
    """Clips a GradList to a global l2 norm of max_norm into its outs; device tensor [norm, S, coef].  out may share
    no memory with the list's tensors."""
    return _grad_list(grads)._call("repro_clip_grad_list", float(max_norm), out, stream)


# The package's __all__ lists the calls of its own file; these are attributes of the package as well.
__all__ = ["GradList", "repro_rope_table", "repro_qk_norm_rope", "repro_qk_norm_rope_backward",
           "repro_grad_list_norm", "repro_clip_grad_list"]
