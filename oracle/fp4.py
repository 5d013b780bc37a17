"""Plain CPU definition of the 4-bit formats, in 64 bits with the roundings to
fp32 that the definition names: e2m1 and e4m3 by nearest member of their value
tables (ties to the even code), no bit tricks, no code shared with the
kernels.  Checks itself against brute force in the tests."""
from __future__ import annotations

import numpy as np

NVFP4, MXFP4 = 0, 1
BLOCK = {NVFP4: 16, MXFP4: 32}

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# e4m3 without sign: codes 0 .. 126 (448); 127 is NaN
E4M3 = np.array([m / 512 for m in range(8)] +
                [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)])[:127]


def nearest(v, table):
    """Index of the member of an ascending non-negative table nearest to |v|,
    ties to the even index, the last member for anything larger."""
    v = np.abs(np.asarray(v, dtype=np.float64))
    hi = np.clip(np.searchsorted(table, v), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = v - table[lo], table[hi] - v
    pick_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    return np.where((v >= table[-1]), len(table) - 1, np.where(pick_lo, lo, hi))


def f32(v):
    with np.errstate(over="ignore", under="ignore", invalid="ignore", divide="ignore"):
        return np.asarray(v, dtype=np.float64).astype(np.float32).astype(np.float64)


def tensor_scale(amax, eps=1e-12):
    """(S, inv) of NVFP4: S = fl32(448 / max(amax, eps)), inv = fl32(1 / S)."""
    s = f32(448.0 / max(float(amax), float(np.float32(eps))))
    with np.errstate(divide="ignore"):
        return float(s), float(f32(1.0 / s))


def blocks(x, fmt):
    rows, cols = x.shape
    b = BLOCK[fmt]
    out = np.zeros((rows, -(-cols // b) * b))
    out[:, :cols] = x
    return out.reshape(rows, -1, b)


def quantise(x, fmt, scale=None):
    """Codes [rows, cols padded to blocks] (4-bit numbers, the sign in bit 3)
    and scale bytes [rows, blocks] of finite x; scale: NVFP4's S."""
    xb = blocks(np.asarray(x, dtype=np.float64), fmt)
    top = np.abs(xb).max(axis=2)
    if fmt == MXFP4:
        _, e = np.frexp(top)
        field = np.where(top >= 2.0 ** -126, e - 1 + 127, 0)
        sc = np.maximum(field - 2, 0)
        v = np.ldexp(xb, (127 - sc)[:, :, None].astype(np.int64))
    else:
        sc = nearest(f32(top * scale), E4M3)
        c = E4M3[sc]
        with np.errstate(divide="ignore", invalid="ignore"):
            r = np.where(c > 0, f32(f32(6.0 * scale) / np.where(c > 0, c, 1.0)), 0.0)
        v = f32(xb * r[:, :, None])
    q = nearest(v, E2M1) | (np.signbit(v).astype(np.int64) << 3)
    return q.reshape(x.shape[0], -1).astype(np.uint8), sc.astype(np.uint8)


def pack(q, cols):
    """Codes -> bytes [rows, ceil(cols / 32) * 16]; codes past cols are zero."""
    rows = q.shape[0]
    full = np.zeros((rows, -(-cols // 32) * 32), np.uint8)
    full[:, :cols] = q[:, :cols]
    return full[:, 0::2] | (full[:, 1::2] << 4)


def tile_scales(sc):
    """Scale bytes [rows, blocks] -> the 512-byte tiles, padding zero."""
    rows, nb = sc.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    out = np.zeros(rt * kt * 512, np.uint8)
    r, k = np.indices(sc.shape)
    at = ((r // 128) * kt + k // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + k % 4
    out[at.ravel()] = sc.ravel()
    return out


def scale_values(sc, fmt):
    sc = sc.astype(np.int64)
    return np.ldexp(1.0, sc - 127) if fmt == MXFP4 else E4M3[sc]


def values(q, sc, fmt, cols, inv=None):
    """What codes and scales stand for, in 64 bits (the factor inv / 6 as fp32)."""
    v = np.where(q & 8, -1.0, 1.0) * E2M1[q & 7]
    v = v.reshape(q.shape[0], -1, BLOCK[fmt]) * scale_values(sc, fmt)[:, :, None]
    v = v.reshape(q.shape[0], -1)[:, :cols]
    return v if fmt == MXFP4 else v * f32(inv / 6.0)
