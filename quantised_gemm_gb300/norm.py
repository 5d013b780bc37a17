"""Layer norm of bf16 rows before a Linear, with the residual that is added
before it, and its backward pass:

  h = bf16(x + residual), or x;  y = (h - mean) * rstd * w + b
  dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dres,  g = dy * w
  dw = sum of dy * xhat, db = sum of dy over the rows,  xhat = (h - mean) * rstd

The output's largest magnitude can be taken on the way, which is what the cast
of the Linear behind it needs, and that of dx for the Linear before it
(link_linears()).  Any row strides and alignments, 1 to 16384 columns;
``include/fp8lin.h`` has the numerics.
"""
from __future__ import annotations

import torch

from . import _lib
from . import Workspace, _dev, _stream
from .fp4 import _matrix

_load = _lib.load

_F32 = {torch.bfloat16: 0, torch.float32: 1}


def _here(*tensors):
    """Refuses tensors of another device than the current one, on whose stream the call runs."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.is_cuda and t.get_device() != dev:
            raise ValueError("a tensor on cuda:%d, but the current device is cuda:%d"
                             % (t.get_device(), dev))


def _param(t: torch.Tensor | None, name: str, cols: int, dtype=None):
    if t is None:
        return None
    if t.dtype not in _F32 or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (name, dtype or "bf16 or fp32", t.dtype))
    if t.dim() != 1 or t.shape[0] != cols or (cols > 1 and t.stride(0) != 1):
        raise ValueError("%s must be contiguous [%d]" % (name, cols))
    return _dev(t, name)


def _rows_like(t: torch.Tensor | None, name: str, rows: int, cols: int):
    """(pointer, row stride) of a bf16 [rows, cols] tensor; (None, 0) for None."""
    if t is None:
        return None, 0
    p, r, c, ld = _matrix(t, name)
    if (r, c) != (rows, cols):
        raise ValueError("%s must be [%d, %d]" % (name, rows, cols))
    return p, ld


def _stats(t: torch.Tensor | None, rows: int):
    if t is None:
        return None
    if tuple(t.shape) != (2, rows) or not t.is_contiguous():
        raise ValueError("stats must be contiguous [2, %d]" % rows)
    return _dev(t, "stats", torch.float32)


def _amax(t: torch.Tensor | None, name: str):
    if t is not None and t.numel() != 1:
        raise ValueError("%s must have one element" % name)
    return _dev(t, name, torch.float32)


def layer_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None, y: torch.Tensor,
               stats: torch.Tensor | None = None, ws: Workspace | None = None, *,
               eps: float = 1e-5, residual: torch.Tensor | None = None,
               h: torch.Tensor | None = None, y_amax: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y = layer norm of x (bf16 [M, K]), or of h = bf16(x + residual), which is
    written too.  w, b: bf16 or fp32 [K]; stats (fp32 [2, M]) receives the rows'
    means and inverse deviations, for the backward; y_amax (fp32[1]) max |y|,
    for which ws is needed.  h may be x or residual, and y may be x or h."""
    px, rows, cols, ldx = _matrix(x, "x")
    _here(x, w, b, y, stats, residual, h, y_amax, None if ws is None else ws.buf)
    if (residual is None) != (h is None):
        raise ValueError("residual and h must be given together")
    if y_amax is not None and ws is None:
        raise ValueError("y_amax needs a Workspace")
    pr, ldr = _rows_like(residual, "residual", rows, cols)
    ph, ldh = _rows_like(h, "h", rows, cols)
    py, ldy = _rows_like(y, "y", rows, cols)
    pw = _param(w, "w", cols)
    st = _load().fp8lin_layer_norm(px, ldx, pr, ldr, ph, ldh, pw, _param(b, "b", cols, w.dtype),
                                   _F32[w.dtype], rows, cols, eps, py, ldy, _stats(stats, rows),
                                   _amax(y_amax, "y_amax"), None if ws is None else ws.ptr,
                                   _stream(stream))
    _lib.check(st, "fp8lin_layer_norm")
    return y


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, stats: torch.Tensor,
                        dx: torch.Tensor | None, dw: torch.Tensor | None, db: torch.Tensor | None,
                        ws: Workspace, *, dres: torch.Tensor | None = None,
                        dx_amax: torch.Tensor | None = None, stream=None):
    """dx, dw and db of the norm whose forward normalised x (its h, where it had
    a residual) and left stats; each may be None.  dres is added to dx: the
    gradient that reaches h past the norm.  dw and db have w's type.  dx may be
    dy or dres."""
    pdy, rows, cols, lddy = _matrix(dy, "dy")
    if ws is None:
        raise ValueError("a Workspace is required")
    _here(dy, x, w, stats, dx, dw, db, dres, dx_amax, ws.buf)
    if dx_amax is not None and dx is None:
        raise ValueError("dx_amax needs dx")
    px, ldx = _rows_like(x, "x", rows, cols)
    pr, ldr = _rows_like(dres, "dres", rows, cols)
    pdx, lddx = _rows_like(dx, "dx", rows, cols)
    pw = _param(w, "w", cols)
    st = _load().fp8lin_layer_norm_backward(
        pdy, lddy, px, ldx, pw, _F32[w.dtype], _stats(stats, rows), rows, cols, pr, ldr, pdx, lddx,
        _param(dw, "dw", cols, w.dtype), _param(db, "db", cols, w.dtype), _amax(dx_amax, "dx_amax"),
        ws.ptr, ws.nbytes, _stream(stream))
    _lib.check(st, "fp8lin_layer_norm_backward")
    return dx, dw, db


class LayerNorm:
    """The buffers of one layer norm of [M, K] tensors: forward(x, w, b) -> y,
    backward(dy) -> (dx, dw, db).  With a residual the sum is kept in ``h`` and
    its gradient past the norm goes into backward(dy, dres).  What the forward
    normalised (x, without a residual) must be unchanged until the backward."""

    def __init__(self, M: int, K: int, *, eps: float = 1e-5, param_dtype=torch.bfloat16,
                 device="cuda"):
        if param_dtype not in _F32:
            raise TypeError("param_dtype must be bf16 or fp32, got %s" % param_dtype)
        self.M, self.K, self.N, self.eps = M, K, K, eps
        bf = dict(dtype=torch.bfloat16, device=device)
        self.y = torch.empty((M, K), **bf)
        self.h = None  # made by the first forward with a residual
        self.dx = torch.empty((M, K), **bf)
        self.dw = torch.empty(K, dtype=param_dtype, device=device)
        self.db = torch.empty(K, dtype=param_dtype, device=device)
        self.stats = torch.empty((2, M), dtype=torch.float32, device=device)
        self.ws = Workspace(M, K, K, device=device)
        # Where max |y| and max |dx| go (set by link_linears()).
        self.y_amax_to = None
        self.dx_amax_to = None
        self._x = self._w = None

    def forward(self, x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None,
                residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        self._x = None
        if w.dtype != self.dw.dtype:
            raise TypeError("w must be %s, got %s" % (self.dw.dtype, w.dtype))
        if residual is not None and self.h is None:
            self.h = torch.empty_like(self.y)
        h = self.h if residual is not None else None
        layer_norm(x, w, b, self.y, self.stats, self.ws, eps=self.eps, residual=residual, h=h,
                   y_amax=self.y_amax_to, stream=stream)
        self._x, self._w = (x if h is None else h), w
        return self.y

    def backward(self, dy: torch.Tensor, dres: torch.Tensor | None = None, need_dx: bool = True,
                 need_dw: bool = True, stream=None):
        """dx, dw and db of the last forward."""
        if self._x is None:
            raise ValueError("no forward has run: there is nothing to differentiate")
        dx, dw, db = (self.dx if need_dx else None), *((self.dw, self.db) if need_dw else (None, None))
        return layer_norm_backward(dy, self._x, self._w, self.stats, dx, dw, db, self.ws, dres=dres,
                                   dx_amax=self.dx_amax_to if need_dx else None, stream=stream)
