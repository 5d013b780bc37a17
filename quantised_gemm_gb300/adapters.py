"""Low-rank adapters of many requests beside a shared Linear, and their
training: row i of a batch has adapter index[i] of a bank, or none.

  h_i = A x_i                         fp32, kept for the backward
  y_i = base_i + s B h_i              base: what the shared weight gave
  dh_i = s B^T dy_i,  dx_i = base_i + A^T dh_i
  dA = sum of dh_i x_i^T,  dB = sum of s dy_i h_i^T   over the adapter's rows

The shared product is fp4_linear(), Fp4Linear, Fp8Linear or any other; its y (or
dx) is the base and may be the output too.  A maximum of the base that the product
delivered to a linked layer (link_linears()) is not that of the output.  Any sizes, row strides and
alignments, ranks up to 128; ``include/fp8lin.h`` has the numerics.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from . import Workspace
from .norm import _current_device, _on, _rows, _rows_like, _stream_on, _whole

_load = _lib.load


class Adapters:
    """A bank of adapters of one Linear: a (bf16 [count, rank, K]), b (bf16
    [count, N, rank]) and scale (fp32 [count]).  An adapter of a smaller rank is
    padded with zeros.  The tensors' values may change between calls (training);
    other tensors take another bank."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor):
        if a.dim() != 3 or b.dim() != 3:
            raise ValueError("a [count, rank, K] and b [count, N, rank] expected")
        count, rank, k = a.shape
        n = b.shape[1]
        c = _lib.AdaptersC()
        self.device = a.get_device()
        c.a = _whole(a, "a", (count, rank, k), torch.bfloat16, self.device)
        c.b = _whole(b, "b", (count, n, rank), torch.bfloat16, self.device)
        c.scale = _whole(scale, "scale", (count,), torch.float32, self.device)
        if self.device < 0:
            raise ValueError("a, b and scale must be CUDA tensors")
        if not (1 <= count <= 1024 and 1 <= rank <= 128 and k >= 1 and n >= 1):
            raise ValueError("1 to 1024 adapters of rank 1 to 128 expected, and K and N of at least 1")
        self._a, self._b, self._scale = a, b, scale
        self.count, self.rank, self.K, self.N = count, rank, k, n
        c.count, c.k, c.n, c.rank = count, k, n, rank
        self._c = c
        self._at = (c.a, c.b, c.scale)
        self._ref = ctypes.byref(c)

    @property
    def a(self) -> torch.Tensor:
        return self._a

    @property
    def b(self) -> torch.Tensor:
        return self._b

    @property
    def scale(self) -> torch.Tensor:
        return self._scale


class AdapterRoute:
    """A batch's rows sorted by adapter, made once by set(index) and given to the
    calls beside every Linear that the batch goes through.  It is for `rows`
    rows and banks of `count` adapters."""

    def __init__(self, rows: int, count: int, device="cuda"):
        self.rows, self.count = rows, count
        nbytes = int(_load().fp8lin_adapter_route_bytes(rows, count))
        if nbytes == 0:
            raise ValueError("0 to 2^24 rows and 1 to 1024 adapters expected")
        self.buf = torch.zeros(nbytes // 4, dtype=torch.int32, device=device)
        self._set = False

    def set(self, index: torch.Tensor, stream=None) -> AdapterRoute:
        dev = _current_device()
        self._set = False
        st = _load().fp8lin_adapter_route(_whole(index, "index", (self.rows,), torch.int32, dev), self.rows,
                                          self.count, _on(self.buf, "the route", dev), _stream_on(dev, stream))
        _lib.check(st, "fp8lin_adapter_route")
        self._set = True
        return self


def _route(route: AdapterRoute | None, rows: int, bank: Adapters, dev: int):
    if route is None:
        return None
    if (route.rows, route.count) != (rows, bank.count):
        raise ValueError("the route is for %d rows and %d adapters, not %d and %d"
                         % (route.rows, route.count, rows, bank.count))
    if not route._set:
        raise ValueError("the route has no index yet")
    return _on(route.buf, "the route", dev)


def _bank(bank: Adapters, dev: int):
    if bank.device != dev:
        raise ValueError("the adapters are on cuda:%d, but the current device is cuda:%d"
                         % (bank.device, dev))
    if (bank._a.data_ptr(), bank._b.data_ptr(), bank._scale.data_ptr()) != bank._at:
        raise ValueError("the bank's tensors have other storage now: make another bank")
    return bank._ref


def _linear_args(x, index, bank, y, h, ws, base, route, stream):
    dev = _current_device()
    px, rows, k, ldx = _rows(x, "x", dev)
    if ws is None:
        raise ValueError("a Workspace is required")
    if k != bank.K:
        raise ValueError("x must be [M, %d]" % bank.K)
    py, ldy = _rows_like(y, "y", rows, bank.N, dev)
    pb, ldb = _rows_like(base, "base", rows, bank.N, dev)
    return (_bank(bank, dev), px, ldx, _whole(index, "index", (rows,), torch.int32, dev),
            _route(route, rows, bank, dev), rows, pb, ldb, py, ldy,
            _whole(h, "h", (rows, bank.rank), torch.float32, dev), _on(ws.buf, "ws", dev), ws.nbytes,
            _stream_on(dev, stream))


def _linear(args):
    _lib.check(_load().fp8lin_adapter_linear(*args), "fp8lin_adapter_linear")


def adapter_linear(x: torch.Tensor, index: torch.Tensor, bank: Adapters, y: torch.Tensor,
                   h: torch.Tensor, ws: Workspace, *, base: torch.Tensor | None = None,
                   route: AdapterRoute | None = None, stream=None) -> torch.Tensor:
    """y = base + the adapters' part for x (bf16 [M, K]).  index: int32 [M], a
    number outside [0, count) for a row without an adapter; base: bf16 [M, N] or
    None for zeros, and may be y; h (fp32 [M, rank]) receives A x, for the
    backward.  route: index sorted before, where several calls share it."""
    _linear(_linear_args(x, index, bank, y, h, ws, base, route, stream))
    return y


def adapter_backward(dy: torch.Tensor, x: torch.Tensor | None, h: torch.Tensor | None,
                     index: torch.Tensor, bank: Adapters, dh: torch.Tensor,
                     dx: torch.Tensor | None, da: torch.Tensor | None, db: torch.Tensor | None,
                     ws: Workspace, *, base: torch.Tensor | None = None,
                     route: AdapterRoute | None = None, stream=None):
    """dx = base + the adapters' part, dA and dB (bf16, of the bank's shapes; zeros
    for adapters that no row has), from the forward's x and h; each of the three
    may be None, x is needed for da only and h for db.  dh: fp32 [M, rank]
    receives s B^T dy, and is not h.  base may be dx."""
    dev = _current_device()
    pdy, rows, n, lddy = _rows(dy, "dy", dev)
    if ws is None:
        raise ValueError("a Workspace is required")
    if n != bank.N:
        raise ValueError("dy must be [M, %d]" % bank.N)
    if (da is not None and x is None) or (db is not None and h is None):
        raise ValueError("da needs x, and db needs h")
    px, ldx = _rows_like(x, "x", rows, bank.K, dev)
    pdx, lddx = _rows_like(dx, "dx", rows, bank.K, dev)
    pb, ldb = _rows_like(base, "base", rows, bank.K, dev)
    low, f32 = (rows, bank.rank), torch.float32
    st = _load().fp8lin_adapter_backward(
        _bank(bank, dev), pdy, lddy, px, ldx, _whole(h, "h", low, f32, dev),
        _whole(index, "index", (rows,), torch.int32, dev), _route(route, rows, bank, dev), rows, pb, ldb,
        pdx, lddx, _whole(dh, "dh", low, f32, dev), _whole(da, "da", bank.a.shape, torch.bfloat16, dev),
        _whole(db, "db", bank.b.shape, torch.bfloat16, dev), _on(ws.buf, "ws", dev), ws.nbytes,
        _stream_on(dev, stream))
    _lib.check(st, "fp8lin_adapter_backward")
    return dx, da, db
