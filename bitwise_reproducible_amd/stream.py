"""The residual stream between two blocks and the loss at its end (binding).

Argument marshalling as in layer.py (OPEN-1B paper, section 3.1: a pre-norm
decoder block with RMS norms; section 3.2: softmax cross entropy and z-loss,
fused and in pieces).  All of these are attributes of the package too:

    repro_residual_norm(x, block=None, gain=None, block_gain=None, gate=None, block_norm=False, x_scale=1.0,
                        block_scale=1.0, eps=1e-6, y=None, out=None) -> (y, out)
    repro_residual_norm_backward(y, block, dy, dout, gain=None, block_gain=None, gate=None, block_norm=False,
                                 x_scale=1.0, block_scale=1.0, eps=1e-6, dx=None, dblock=None, dgain=None,
                                 dblock_gain=None, dgate=None, workspace=None)
        -> (dx, dblock, dgain, dblock_gain, dgate)
    repro_vocab_loss(x, weight, labels, z_weight=0.0, ignore_index=-100, loss=None, lse=None, workspace=None)
        -> (loss, lse)
    repro_vocab_loss_backward(x, weight, labels, lse, dloss, z_weight=0.0, ignore_index=-100, dx=None, dweight=None,
                              workspace=None) -> (dx, dweight)

Rows are (dim), (rows, dim) or (batch, seq, dim) tensors of float32 or bfloat16
with any strides of the first two dimensions; the loss takes (tokens, dim) and
(vocab, dim) matrices with any distance between rows.  No output may share
memory with another tensor of its call, but for the norm's rows over an input of
the very same view.
`stream` orders everything a call does, its own allocations too; without it
that is the current stream.  As with the package's other calls, autograd
records none of them: the backward pass is a call of its own.
"""
from __future__ import annotations

import ctypes

import torch

from bitwise_reproducible_amd import layer as _layer

_calls = None


def _lib():
    """The library, with these entry points' argument types set."""
    lib = _layer._lib()
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    lib.repro_residual_norm.argtypes = [vp, vp]
    lib.repro_residual_workspace_bytes.argtypes = [vp]
    lib.repro_residual_workspace_bytes.restype = i64
    lib.repro_residual_norm_backward.argtypes = [vp, vp, i64, vp]
    for name in ("repro_vocab_loss", "repro_vocab_loss_backward"):
        getattr(lib, name).argtypes = [vp, vp, i64, vp]
        size = getattr(lib, name + "_workspace_bytes")
        size.argtypes, size.restype = [vp], i64
    for name in ("repro_residual_norm", "repro_residual_norm_backward", "repro_vocab_loss",
                 "repro_vocab_loss_backward"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


def _load():
    """layer.py's extension, with these entry points bound."""
    global _calls
    if _calls is None:
        module, lib = _layer._load(), _lib()
        module.bind_stream(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "repro_residual_norm", "repro_residual_workspace_bytes", "repro_residual_norm_backward",
            "repro_vocab_loss_workspace_bytes", "repro_vocab_loss", "repro_vocab_loss_backward_workspace_bytes",
            "repro_vocab_loss_backward")))
        _calls = module
    return _calls


def repro_residual_norm(x, block=None, gain=None, block_gain=None, gate=None, block_norm: bool = False,
                        x_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6, y=None, out=None,
                        stream=None):
    """(y, out): y = x_scale * x + block_scale * gate * block, the block's output normed first with block_norm (and
    scaled by block_gain), and out = the norm of y times gain.  gate is of the rows' shape and type, or, where the rows
    have more dimensions than (dim), a (dim) vector for the channels, of the gains' type.
    Without a block out is the norm of x, y is None, and the scales have to be 1, here and in the backward pass (see
    repro.h)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_residual_norm(x, block, gain, block_gain, gate, block_norm, x_scale, block_scale, eps, y, out)
    return _layer._done((_calls or _load()).residual(x, block, gain, block_gain, gate, block_norm, x_scale,
                                                     block_scale, eps, y, out), "repro_residual_norm")


def repro_residual_norm_backward(y, block, dy, dout, gain=None, block_gain=None, gate=None, block_norm: bool = False,
                                 x_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6, dx=None,
                                 dblock=None, dgain=None, dblock_gain=None, dgate=None, workspace=None, stream=None):
    """Gradients of repro_residual_norm at its y and block for the gradients dy of y (None: none) and dout of out:
    (dx, dblock, dgain, dblock_gain, dgate).  Those of gains and of a gate for the channels are float32, that of a gate
    of the rows' shape (a row of its own, (dim), has no other) is of the rows' type; each is None where there is nothing
    that it is the gradient of.  Where the block reaches the sum as it is, with the scale of x,
    and no dblock is given, dblock is dx itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_residual_norm_backward(y, block, dy, dout, gain, block_gain, gate, block_norm, x_scale,
                                                block_scale, eps, dx, dblock, dgain, dblock_gain, dgate, workspace)
    return _layer._done((_calls or _load()).residual_backward(
        y, block, dy, dout, gain, block_gain, gate, block_norm, x_scale, block_scale, eps, dx, dblock, dgain,
        dblock_gain, dgate, workspace), "repro_residual_norm_backward")


def repro_vocab_loss(x, weight, labels, z_weight: float = 0.0, ignore_index: int = -100, loss=None, lse=None,
                     workspace=None, stream=None):
    """(loss, lse) of each token, float32: loss = lse - logit[label] + z_weight * lse^2 with the logits x weight^T and
    lse the logarithm of the sum of their exponentials; 0 where the label is ignore_index, NaN where it is outside the
    vocabulary (see repro.h).  An entry whose logit is -inf counts for nothing in bfloat16; in float32 a weight of -inf,
    or of 2^128 (1 - 2^-9) and more in size, makes the loss NaN, as its product is one of three parts."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_vocab_loss(x, weight, labels, z_weight, ignore_index, loss, lse, workspace)
    return _layer._done((_calls or _load()).loss(x, weight, labels, z_weight, ignore_index, loss, lse, workspace),
                        "repro_vocab_loss")


def repro_vocab_loss_backward(x, weight, labels, lse, dloss, z_weight: float = 0.0, ignore_index: int = -100, dx=None,
                              dweight=None, workspace=None, stream=None):
    """(dx, dweight) of repro_vocab_loss for the losses' gradients dloss, float32: one for each token, or one number
    (a tensor without dimensions) for all of them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return repro_vocab_loss_backward(x, weight, labels, lse, dloss, z_weight, ignore_index, dx, dweight,
                                             workspace)
    return _layer._done((_calls or _load()).loss_backward(x, weight, labels, lse, dloss, z_weight, ignore_index, dx,
                                                          dweight, workspace), "repro_vocab_loss_backward")


# The package's __all__ lists the calls of its own file; these are attributes of the package as well.
__all__ = ["repro_residual_norm", "repro_residual_norm_backward", "repro_vocab_loss", "repro_vocab_loss_backward"]
