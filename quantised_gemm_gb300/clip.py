"""The global 2-norm of a list of gradients and their clipping to a largest
norm, as a training step does after its backwards:

  norm = sqrt(sum over all tensors of g^2),  g <- g * min(1, max_norm / (norm + eps))

The norm stays on the device.  Gradients may be bf16 or fp32, mixed, of any
size; a data-parallel program reduces the squares over its ranks between
grad_norm() and clip_grads().
"""
from __future__ import annotations

import array

import torch

from . import _lib
from . import Workspace, _stream

_load = _lib.load


def _same_dense(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the elements of a and b lie without gaps and in the same order."""
    if a.is_contiguous() and b.is_contiguous():
        return True
    want = 1
    for size, stride in sorted(((s, t) for s, t in zip(a.shape, a.stride()) if s != 1),
                               key=lambda v: v[1]):
        if stride != want:
            return False
        want *= size
    return all(s == 1 or t == u for s, t, u in zip(a.shape, a.stride(), b.stride()))


_F32 = {torch.bfloat16: 0, torch.float32: 1}


def _list(grads, outs):
    """(array of fp8lin_grad, as 64-bit words; its length; the outputs)."""
    grads = list(grads)
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError("outs must have one tensor for each gradient")
    words = array.array("Q")  # g, out, n, g_f32 | out_f32 << 32
    for g, o in zip(grads, outs):
        f32 = _F32.get(g.dtype)
        of32 = f32 if o is g else _F32.get(o.dtype)
        if f32 is None or of32 is None:
            raise TypeError("gradients must be bf16 or fp32, got %s, %s" % (g.dtype, o.dtype))
        if not (g.is_cuda and (o is g or o.is_cuda)):
            raise ValueError("gradients must be CUDA tensors")
        if o is not g and o.shape != g.shape:
            raise ValueError("an output must have its gradient's shape")
        if not (g.is_contiguous() and (o is g or o.is_contiguous())) and not _same_dense(g, o):
            raise ValueError("a gradient must be dense, and its output in the same order")
        at = g.data_ptr()
        words.extend((at, at if o is g else o.data_ptr(), g.numel(), f32 | of32 << 32))
    return words, len(grads), outs


def _norm_ptr(norm: torch.Tensor) -> int:
    if not norm.is_cuda or norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be a CUDA fp32 tensor of one element")
    return norm.data_ptr()


def grad_norm(grads, norm: torch.Tensor, ws: Workspace, stream=None) -> torch.Tensor:
    """norm (fp32[1]) = the 2-norm of all gradients together."""
    arr, n, _ = _list(grads, None)
    _lib.check(_load().fp8lin_grad_norm(arr.buffer_info()[0], n, _norm_ptr(norm), ws.ptr,
                                        ws.nbytes, _stream(stream)), "fp8lin_grad_norm")
    return norm


def clip_grads(grads, max_norm: float, norm: torch.Tensor, *, outs=None, eps: float = 1e-6,
               stream=None):
    """Scale every gradient by min(1, max_norm / (norm + eps)), in place or
    into outs (bf16 or fp32, e.g. an optimizer's fp32 buffers)."""
    arr, n, outs = _list(grads, outs)
    _lib.check(_load().fp8lin_grad_clip(arr.buffer_info()[0], n, _norm_ptr(norm), max_norm, eps,
                                        _stream(stream)), "fp8lin_grad_clip")
    return outs


def clip_grad_norm(grads, max_norm: float, norm: torch.Tensor, ws: Workspace, *, outs=None,
                   eps: float = 1e-6, stream=None) -> torch.Tensor:
    """grad_norm() and clip_grads() in one call; returns the norm before
    clipping (on the device)."""
    arr, n, _ = _list(grads, outs)
    st = _load().fp8lin_grad_clip_norm(arr.buffer_info()[0], n, max_norm, eps, _norm_ptr(norm),
                                       ws.ptr, ws.nbytes, _stream(stream))
    _lib.check(st, "fp8lin_grad_clip_norm")
    return norm
