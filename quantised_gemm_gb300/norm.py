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
from . import Workspace, _raw_stream, _stream

_load = _lib.load

_BF16 = torch.bfloat16
_F32 = {torch.bfloat16: 0, torch.float32: 1}
_current_device = torch._C._cuda_getDevice


def _stream_on(dev: int, stream) -> int:
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _on(t: torch.Tensor, name: str, dev: int):
    """Refuses a tensor of another device than the current one, on whose stream the call runs."""
    at = t.get_device()
    if at != dev:
        raise ValueError("%s must be a CUDA tensor" % name if at < 0 else
                         "%s is on cuda:%d, but the current device is cuda:%d" % (name, at, dev))
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dev: int):
    """(pointer, rows, cols, row stride) of a 2-D bf16 tensor with unit column stride."""
    if t.dtype is not _BF16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError("%s must have unit column stride" % name)
    if ld < cols:
        if rows > 1:
            raise ValueError("%s must not have overlapping rows" % name)
        ld = cols
    return _on(t, name, dev), rows, cols, ld


def _rows_like(t: torch.Tensor | None, name: str, rows: int, cols: int, dev: int):
    """(pointer, row stride) of a bf16 [rows, cols] tensor; (None, 0) for None."""
    if t is None:
        return None, 0
    p, r, c, ld = _rows(t, name, dev)
    if r != rows or c != cols:
        raise ValueError("%s must be [%d, %d]" % (name, rows, cols))
    return p, ld


def _whole(t: torch.Tensor | None, name: str, shape, dtype, dev: int):
    """The pointer of a contiguous tensor of this shape and type; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous %s" % (name, list(shape)))
    return _on(t, name, dev)


def _amax(t: torch.Tensor | None, name: str, dev: int):
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.numel() != 1:
        raise ValueError("%s must be fp32 with one element" % name)
    return _on(t, name, dev)


def layer_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor | None, y: torch.Tensor,
               stats: torch.Tensor | None = None, ws: Workspace | None = None, *,
               eps: float = 1e-5, residual: torch.Tensor | None = None,
               h: torch.Tensor | None = None, y_amax: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y = layer norm of x (bf16 [M, K]), or of h = bf16(x + residual), which is
    written too.  w, b: bf16 or fp32 [K]; stats (fp32 [2, M]) receives the rows'
    means and inverse deviations, for the backward; y_amax (fp32[1]) max |y|,
    for which ws is needed.  h may be x or residual, and y may be any of the three."""
    dev = _current_device()
    px, rows, cols, ldx = _rows(x, "x", dev)
    if (residual is None) != (h is None):
        raise ValueError("residual and h must be given together")
    if y_amax is not None and ws is None:
        raise ValueError("y_amax needs a Workspace")
    f32 = _F32.get(w.dtype)
    if f32 is None:
        raise TypeError("w must be bf16 or fp32, got %s" % w.dtype)
    pr, ldr = _rows_like(residual, "residual", rows, cols, dev)
    ph, ldh = _rows_like(h, "h", rows, cols, dev)
    py, ldy = _rows_like(y, "y", rows, cols, dev)
    pw = _whole(w, "w", (cols,), w.dtype, dev)
    pb = _whole(b, "b", (cols,), w.dtype, dev)
    st = _load().fp8lin_layer_norm(px, ldx, pr, ldr, ph, ldh, pw, pb, f32, rows, cols, eps, py, ldy,
                                   _whole(stats, "stats", (2, rows), torch.float32, dev),
                                   _amax(y_amax, "y_amax", dev),
                                   None if ws is None else _on(ws.buf, "ws", dev), _stream_on(dev, stream))
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
    dev = _current_device()
    pdy, rows, cols, lddy = _rows(dy, "dy", dev)
    if ws is None:
        raise ValueError("a Workspace is required")
    if dx_amax is not None and dx is None:
        raise ValueError("dx_amax needs dx")
    if stats is None:
        raise ValueError("stats is required")
    dtype = w.dtype
    f32 = _F32.get(dtype)
    if f32 is None:
        raise TypeError("w must be bf16 or fp32, got %s" % dtype)
    px, ldx = _rows_like(x, "x", rows, cols, dev)
    pr, ldr = _rows_like(dres, "dres", rows, cols, dev)
    pdx, lddx = _rows_like(dx, "dx", rows, cols, dev)
    one = (cols,)
    st = _load().fp8lin_layer_norm_backward(
        pdy, lddy, px, ldx, _whole(w, "w", one, dtype, dev), f32,
        _whole(stats, "stats", (2, rows), torch.float32, dev), rows, cols, pr, ldr, pdx, lddx,
        _whole(dw, "dw", one, dtype, dev), _whole(db, "db", one, dtype, dev),
        _amax(dx_amax, "dx_amax", dev), _on(ws.buf, "ws", dev), ws.nbytes, _stream_on(dev, stream))
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
