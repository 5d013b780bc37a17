"""The global 2-norm of a list of gradients and their clipping to a largest
norm, as a training step does after its backwards:

  norm = sqrt(sum over all tensors of g^2),  g <- g * min(1, max_norm / (norm + eps))

The norm stays on the device.  Gradients may be bf16 or fp32, mixed, of any
size; a data-parallel program reduces the squares over its ranks between
grad_norm() and clip_grads().
"""
from __future__ import annotations

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


def _list(grads, outs):
    grads = [g for g in grads]
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError("outs must have one tensor for each gradient")
    arr = (_lib.GradC * max(1, len(grads)))()
    for i, (g, o) in enumerate(zip(grads, outs)):
        if not g.is_cuda or not o.is_cuda:
            raise ValueError("gradients must be CUDA tensors")
        f32, of32 = g.dtype == torch.float32, o.dtype == torch.float32
        if not (f32 or g.dtype == torch.bfloat16) or not (of32 or o.dtype == torch.bfloat16):
            raise TypeError("gradients must be bf16 or fp32, got %s, %s" % (g.dtype, o.dtype))
        if o is not g and o.shape != g.shape:
            raise ValueError("an output must have its gradient's shape")
        if not _same_dense(g, o):
            raise ValueError("a gradient must be dense, and its output in the same order")
        c = arr[i]
        c.g, c.out, c.n = g.data_ptr(), o.data_ptr(), g.numel()
        c.g_f32, c.out_f32 = f32, of32
    return arr, len(grads), outs


def _norm_ptr(norm: torch.Tensor) -> int:
    if not norm.is_cuda or norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be a CUDA fp32 tensor of one element")
    return norm.data_ptr()


def grad_norm(grads, norm: torch.Tensor, ws: Workspace, stream=None) -> torch.Tensor:
    """norm (fp32[1]) = the 2-norm of all gradients together."""
    arr, n, _ = _list(grads, None)
    _lib.check(_load().fp8lin_grad_norm(arr, n, _norm_ptr(norm), ws.ptr, ws.nbytes,
                                        _stream(stream)), "fp8lin_grad_norm")
    return norm


def clip_grads(grads, max_norm: float, norm: torch.Tensor, *, outs=None, eps: float = 1e-6,
               stream=None):
    """Scale every gradient by min(1, max_norm / (norm + eps)), in place or
    into outs (bf16 or fp32, e.g. an optimizer's fp32 buffers)."""
    arr, n, outs = _list(grads, outs)
    _lib.check(_load().fp8lin_grad_clip(arr, n, _norm_ptr(norm), max_norm, eps, _stream(stream)),
               "fp8lin_grad_clip")
    return outs


def clip_grad_norm(grads, max_norm: float, norm: torch.Tensor, ws: Workspace, *, outs=None,
                   eps: float = 1e-6, stream=None) -> torch.Tensor:
    """grad_norm() and clip_grads() in one call; returns the norm before
    clipping (on the device)."""
    arr, n, _ = _list(grads, outs)
    _lib.check(_load().fp8lin_grad_clip_norm(arr, n, max_norm, eps, _norm_ptr(norm), ws.ptr,
                                             ws.nbytes, _stream(stream)), "fp8lin_grad_clip_norm")
    return norm
