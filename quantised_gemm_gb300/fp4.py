"""Microscaled 4-bit operands: tensors in NVFP4 or MXFP4, their quantisation
from bf16, the products of two of them, and a Linear whose forward and
backward run in 4 bits.

  NVFP4  e2m1 values in blocks of 16 with an e4m3 scale, and one fp32 scale a
         tensor: the e4m3 ScalingState of the 8-bit path, so dynamic, delayed
         and precomputed scaling apply as they do there.
  MXFP4  e2m1 values in blocks of 32 with a power-of-two scale; no state.

The blocks run along a row, the axis a product contracts over.  A backward
contracts over the other one, so quantisation writes a second, transposed
copy with its own blocks in the same read.  Any sizes, row strides and
alignments are taken; ``include/fp8lin.h`` has the layout and the numerics.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from . import (AMAX_AUTO, DELAYED, DYNAMIC, E4M3, MXFP4, NVFP4, ScalingState, Workspace, _dev,
               _stream, scale_many)
from .adapters import AdapterRoute, Adapters, _linear, _linear_args

_load = _lib.load


class Fp4Tensor:
    """A [rows, cols] tensor in 4 bits.

    codes: uint8 [rows, ceil(cols / 32) * 16]; scales: uint8, 512-byte tiles
    of 128 rows x 4 blocks.  Both are allocated (zero) unless given.  An NVFP4
    tensor is quantised with ``state`` (made here unless given; a tensor and
    its transposed copy share one) and keeps the inverse scale that its codes
    were made with in ``inv_scale`` (fp32[1]), so it may be used after the
    state has moved on.  A tensor that is only read is given ``inv_scale``
    instead of a state."""

    def __init__(self, rows: int, cols: int, fmt: int = NVFP4, *, state: ScalingState | None = None,
                 codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                 inv_scale: torch.Tensor | None = None, device="cuda"):
        if fmt not in (NVFP4, MXFP4):
            raise ValueError("fmt must be NVFP4 or MXFP4")
        if rows < 0 or cols < 0:
            raise ValueError("rows and cols must not be negative")
        self.rows, self.cols, self.fmt = rows, cols, fmt
        if fmt == MXFP4 and (state is not None or inv_scale is not None):
            raise ValueError("MXFP4 has no tensorwise scale")
        if state is not None and inv_scale is not None:
            raise ValueError("give state or inv_scale, not both")
        ld = (cols + 31) // 32 * 16
        nbytes = int(_load().fp8lin_fp4_scale_bytes(rows, cols, fmt))
        if codes is None:
            codes = torch.zeros((rows, ld), dtype=torch.uint8, device=device)
        if scales is None:
            scales = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        if codes.dim() != 2 or codes.shape[0] != rows or codes.shape[1] < ld or \
                (codes.numel() and codes.stride(1) != 1):
            raise ValueError("codes must be [%d, >= %d] with unit column stride" % (rows, ld))
        if scales.numel() < nbytes or not scales.is_contiguous():
            raise ValueError("scales must be contiguous, at least %d bytes" % nbytes)
        if fmt == NVFP4 and state is None and inv_scale is None:
            state = ScalingState(E4M3, DYNAMIC, amax_algo=AMAX_AUTO, device=codes.device)
        self.state = state
        self.inv_scale = state.inv_scale.clone() if state is not None else inv_scale
        if self.inv_scale is not None and self.inv_scale.numel() != 1:
            raise ValueError("inv_scale must have one element")
        self._codes, self._scales = codes, scales
        c = _lib.Fp4TensorC()
        c.codes, c.scales = _dev(codes, "codes", torch.uint8), _dev(scales, "scales", torch.uint8)
        if state is not None:
            c.inv_scale = _dev(state.inv_scale, "inv_scale", torch.float32)
            c.own_inv = self.inv_scale.data_ptr()
        else:
            c.inv_scale = _dev(self.inv_scale, "inv_scale", torch.float32)
        c.rows, c.cols, c.ld, c.fmt = rows, cols, (codes.stride(0) if rows > 1 else codes.shape[1]), fmt
        self._c = c
        self._ref = ctypes.byref(c)

    @property
    def codes(self) -> torch.Tensor:
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        return self._scales


def _matrix(t: torch.Tensor, name: str, dtype=torch.bfloat16):
    """(pointer, rows, cols, row stride) of a 2-D CUDA tensor with unit column stride."""
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
    return _dev(t, name, dtype), rows, cols, ld


def _dense(t: torch.Tensor, name: str, rows: int, cols: int):
    if t.shape != (rows, cols) or not t.is_contiguous():
        raise ValueError("%s must be contiguous [%d, %d]" % (name, rows, cols))
    return _dev(t, name, torch.bfloat16)


def _ref(t: Fp4Tensor | None):
    return None if t is None else t._ref


def _state_arg(state: ScalingState | None):
    return None if state is None else ctypes.byref(state.c_struct())


def _source_state(x4: Fp4Tensor) -> ScalingState | None:
    if x4.fmt == NVFP4 and x4.state is None:
        raise ValueError("an NVFP4 tensor without a ScalingState cannot be quantised into")
    return x4.state


def fp4_quantise(x: torch.Tensor, out: Fp4Tensor | None, out_t: Fp4Tensor | None = None,
                 ws: Workspace | None = None, stream=None):
    """Quantise x (bf16 [rows, cols], unit column stride) into out, and into
    out_t ([cols, rows]) the transposed copy; either may be None.  NVFP4 scales
    by the tensors' ScalingState (one state for both)."""
    t = out if out is not None else out_t
    if t is None:
        raise ValueError("out or out_t is required")
    if ws is None:
        raise ValueError("a Workspace is required")
    if out is not None and out_t is not None and out.state is not out_t.state:
        raise ValueError("out and out_t must share one ScalingState")
    px, rows, cols, ld = _matrix(x, "x")
    state = _source_state(t)
    st = _load().fp8lin_fp4_quantise(px, rows, cols, ld, _state_arg(state), _ref(out), _ref(out_t),
                                     ws.ptr, _stream(stream))
    if state is not None:
        state._pull()
    _lib.check(st, "fp8lin_fp4_quantise")
    return out


def fp4_dequantise(t: Fp4Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """The values t stands for, into out ([rows, cols], bf16 or fp32)."""
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("out must be bf16 or fp32, got %s" % out.dtype)
    po, rows, cols, ldo = _matrix(out, "out", out.dtype)
    if (rows, cols) != (t.rows, t.cols):
        raise ValueError("out must be [%d, %d]" % (t.rows, t.cols))
    st = _load().fp8lin_fp4_dequantise(t._ref, po, ldo, 1 if out.dtype == torch.float32 else 0,
                                       _stream(stream))
    _lib.check(st, "fp8lin_fp4_dequantise")
    return out


def _product_out(out: torch.Tensor, name: str, rows: int, cols: int):
    po, r, c, ldo = _matrix(out, name)
    if r != rows or c != cols:
        raise ValueError("%s must be [%d, %d]" % (name, rows, cols))
    return po, ldo


def fp4_gemm(a: Fp4Tensor, b: Fp4Tensor, out: torch.Tensor, ws: Workspace,
             stream=None) -> torch.Tensor:
    """out[m, n] = bf16(sum_k a[m, k] b[n, k]) with fp32 accumulation; a and b
    in the same format, out bf16 with unit column stride."""
    po, ldo = _product_out(out, "out", a.rows, b.rows)
    st = _load().fp8lin_fp4_gemm(a._ref, b._ref, po, ldo, ws.ptr, ws.nbytes, _stream(stream))
    _lib.check(st, "fp8lin_fp4_gemm")
    return out


def fp4_linear(x: torch.Tensor, x4: Fp4Tensor, w4: Fp4Tensor, y: torch.Tensor, ws: Workspace,
               stream=None, *, adapters: Adapters | None = None, index: torch.Tensor | None = None,
               h: torch.Tensor | None = None, route: AdapterRoute | None = None) -> torch.Tensor:
    """y = x W^T for a weight kept in 4 bits: x is quantised into x4, then
    multiplied with w4.  With adapters, y += the part of each row's adapter as
    adapter_linear(x, index, adapters, y, h, ws, base=y, route=route) adds it."""
    px, rows, cols, ld = _matrix(x, "x")
    if rows != x4.rows or cols != x4.cols:
        raise ValueError("x4 must be [%d, %d]" % (rows, cols))
    py, ldy = _product_out(y, "y", rows, w4.rows)
    if (adapters is None) != (index is None) or (adapters is None) != (h is None):
        raise ValueError("adapters, index and h must be given together")
    if route is not None and adapters is None:
        raise ValueError("a route needs adapters")
    low = None
    if adapters is not None:
        low = _linear_args(x, index, adapters, y, h, ws, y, route, stream)
    state = _source_state(x4)
    st = _load().fp8lin_fp4_linear(px, ld, _state_arg(state), x4._ref, w4._ref, py, ldy, ws.ptr,
                                   ws.nbytes, _stream(stream))
    if state is not None:
        state._pull()
    _lib.check(st, "fp8lin_fp4_linear")
    if low is not None:
        _linear(low)
    return y


class Fp4Linear:
    """One Linear y = x W^T with x [M, K], W [N, K] whose three products run in
    4 bits, as Fp8Linear's run in 8: forward(x, w), backward(dy) -> (dX, dW),
    sync_scales() for delayed scaling.  Any M, K, N."""

    def __init__(self, M: int, K: int, N: int, *, fmt: int = NVFP4, scaling: str = "dynamic",
                 history_len: int = 16, amax_algo: int = AMAX_AUTO, eps: float = 1e-12,
                 device="cuda"):
        kind = {"dynamic": DYNAMIC, "delayed": DELAYED}[scaling]
        if fmt == MXFP4 and kind == DELAYED:
            raise ValueError("MXFP4 has no tensorwise scale to delay")
        self.M, self.K, self.N, self.fmt = M, K, N, fmt

        def pair(rows, cols):
            st = ScalingState(E4M3, kind, history_len, amax_algo, eps, device) \
                if fmt == NVFP4 else None
            return (Fp4Tensor(rows, cols, fmt, state=st, device=device),
                    Fp4Tensor(cols, rows, fmt, state=st, device=device))

        self.x4, self.x4t = pair(M, K)
        self.w4, self.w4t = pair(N, K)
        self.dy4, self.dy4t = pair(M, N)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.y = torch.empty((M, N), **bf)
        self.dx = torch.empty((M, K), **bf)
        self.dw = torch.empty((N, K), **bf)
        self.ws = Workspace(M, K, N, device=device)
        self.sx, self.sw, self.sdy = self.x4.state, self.w4.state, self.dy4.state
        self._has_w = False  # w4 and w4t hold a weight at sw's scale
        self._has_x = False  # x4t and w4t hold what a forward multiplied

    def forward(self, x: torch.Tensor, w: torch.Tensor | None, stream=None) -> torch.Tensor:
        """y = x W^T; w = None: the weight of the last forward that was given
        one, without quantising it again (micro-batches of one step)."""
        px = _dense(x, "x", self.M, self.K)
        if w is None and not self._has_w:
            raise ValueError("w is required: no weight has been quantised at the present scale")
        pw = None if w is None else _dense(w, "w", self.N, self.K)
        st = _load().fp8lin_fp4_forward(
            px, pw, _state_arg(self.sx), _state_arg(self.sw), self.x4._ref, self.x4t._ref,
            self.w4._ref, self.w4t._ref, self.y.data_ptr(), self.ws.ptr, self.ws.nbytes,
            _stream(stream))
        for s in (self.sx, self.sw):
            if s is not None:
                s._pull()
        if w is not None:
            self._has_w = st == 0
        self._has_x = st == 0
        _lib.check(st, "fp8lin_fp4_forward")
        return self.y

    def backward(self, dy: torch.Tensor, need_dx: bool = True, need_dw: bool = True, stream=None):
        """dX and dW of the last forward."""
        if not self._has_x:
            raise ValueError("no forward has run: there is nothing to differentiate")
        st = _load().fp8lin_fp4_backward(
            _dense(dy, "dy", self.M, self.N), _state_arg(self.sdy), self.dy4._ref, self.dy4t._ref,
            self.w4t._ref, self.x4t._ref, self.dx.data_ptr() if need_dx else None,
            self.dw.data_ptr() if need_dw else None, self.ws.ptr, self.ws.nbytes, _stream(stream))
        if self.sdy is not None:
            self.sdy._pull()
        _lib.check(st, "fp8lin_fp4_backward")
        return (self.dx if need_dx else None), (self.dw if need_dw else None)

    def sync_scales(self, stream=None):
        """Delayed scaling: push this step's amaxes into the histories and
        recompute the scales; the next forward needs its weight again."""
        delayed = [s for s in (self.sx, self.sw, self.sdy) if s is not None and s.kind == DELAYED]
        if delayed:
            scale_many(delayed, stream)
            self._has_w = False

    def step(self, x, w, dy, stream=None):
        """One forward + backward (+ delayed sync)."""
        self.forward(x, w, stream)
        self.backward(dy, stream=stream)
        self.sync_scales(stream)
        return self.y, self.dx, self.dw
