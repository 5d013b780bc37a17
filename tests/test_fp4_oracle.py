"""The 4-bit oracle against the format definitions, by brute force, and the
argument checks of the 4-bit and gradient calls (no GPU needed)."""
import ctypes

import numpy as np
import pytest

from oracle import fp4 as o4


def test_tables():
    assert len(o4.E2M1) == 8 and o4.E2M1[-1] == 6
    assert len(o4.E4M3) == 127 and o4.E4M3[-1] == 448 and o4.E4M3[1] == 2.0 ** -9
    assert np.all(np.diff(o4.E4M3) > 0)


@pytest.mark.parametrize("table", [o4.E2M1, o4.E4M3], ids=["e2m1", "e4m3"])
def test_nearest_is_the_nearest_and_ties_go_to_even(table):
    mids = (table[1:] + table[:-1]) / 2
    for i, m in enumerate(mids):
        even = i if i % 2 == 0 else i + 1
        assert o4.nearest(m, table) == even
        assert o4.nearest(np.nextafter(m, 0), table) == i
        assert o4.nearest(np.nextafter(m, 1e9), table) == i + 1
    g = np.random.default_rng(3).uniform(0, table[-1] * 1.2, 2000)
    want = [int(np.argmin(np.abs(table - v))) for v in g]  # no exact tie among these
    assert np.array_equal(o4.nearest(g, table), want)


@pytest.mark.parametrize("fmt", [o4.NVFP4, o4.MXFP4])
def test_error_of_a_block_is_bounded(fmt):
    # Half the widest step of e2m1 (2 of 6) and the rounding of the block's
    # scale bound a value's error by a fixed share of the block's maximum:
    # NVFP4 1 / 6 * (1 + 1 / 16) of it plus saturation 1 / 16, MXFP4 by a quarter.
    x = np.random.default_rng(5).normal(size=(64, 128)).astype(np.float32)
    x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    s, inv = o4.tensor_scale(np.abs(x).max())
    q, sc = o4.quantise(x, fmt, s)
    v = o4.values(q, sc, fmt, 128, inv)
    top = np.abs(o4.blocks(x, fmt)).max(axis=2).repeat(o4.BLOCK[fmt], axis=1)
    assert np.all(np.abs(v - x) <= 0.25 * top + 1e-12)


def test_mx_scale_is_the_exponent_less_two():
    x = np.zeros((4, 32))
    x[0, 3], x[1, 0], x[2, 31] = 6.0, -1.0, 2.0 ** -126
    q, sc = o4.quantise(x, o4.MXFP4)
    assert sc[:, 0].tolist() == [127, 125, 0, 0]
    assert q[0, 3] == 7 and q[1, 0] == 8 + 6 and q[2, 31] == 4  # 6, -4 * 2^-2, 2 * 2^-127


def test_layouts():
    sc = np.arange(130 * 5).reshape(130, 5) % 251
    t = o4.tile_scales(sc.astype(np.uint8))
    assert t.size == 2 * 2 * 512
    assert t[0] == sc[0, 0] and t[3] == sc[0, 3] and t[4] == sc[32, 0] and t[16] == sc[1, 0]
    assert t[512] == sc[0, 4] and t[1024 + 16 + 1] == sc[129, 1]
    q = np.arange(33).reshape(1, 33).astype(np.uint8) % 16
    p = o4.pack(q, 33)
    assert p.shape == (1, 32) and p[0, 0] == 0x10 and p[0, 16] == 0 and p[0, 17] == 0


# ---------------------------------------------------------------- arguments


@pytest.fixture(scope="module")
def lib():
    from quantised_gemm_gb300 import build as qb
    qb.build()
    import quantised_gemm_gb300 as q
    return q.library()


def _t4(rows, cols, fmt=0, **kw):
    import quantised_gemm_gb300._lib as L
    c = L.Fp4TensorC()
    c.codes, c.scales, c.inv_scale = 0x10000, 0x20000, 0x30000 if fmt == 0 else None
    c.rows, c.cols, c.ld, c.fmt = rows, cols, (cols + 31) // 32 * 16, fmt
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _state(**kw):
    import quantised_gemm_gb300._lib as L
    s = L.ScalingStateC()
    s.amax = s.scale = 0x40000
    s.inv_scale = 0x30000
    s.history_len, s.fmt, s.kind, s.amax_algo, s.eps = 1, 0, 0, 0, 1e-12
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_scale_bytes(lib):
    for rows, cols, fmt in ((1, 1, 0), (128, 64, 0), (129, 65, 0), (1009, 1531, 1), (0, 5, 0)):
        nb = -(-cols // o4.BLOCK[fmt])
        assert lib.fp8lin_fp4_scale_bytes(rows, cols, fmt) == -(-rows // 128) * -(-nb // 4) * 512
    assert lib.fp8lin_fp4_scale_bytes(-1, 4, 0) == 0 and lib.fp8lin_fp4_scale_bytes(4, 4, 2) == 0


def test_quantise_refusals(lib):
    import quantised_gemm_gb300._lib as L
    p, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    ref = lambda c: None if c is None else ctypes.byref(c)  # noqa: E731

    def call(out, out_t=None, st=_state(), x=p, rows=16, cols=48, ld=48, w=ws):
        return lib.fp8lin_fp4_quantise(x, rows, cols, ld, ref(st), ref(out), ref(out_t), w, None)

    ok = _t4(16, 48)
    assert call(None) == L.EINVAL                                  # no destination
    assert call(ok, w=None) == L.EINVAL                            # no workspace
    assert call(ok, x=None) == L.EINVAL
    assert call(ok, x=ctypes.c_void_p(0x100001)) == L.EINVAL       # odd address
    assert call(ok, ld=40) == L.EINVAL                             # rows overlap
    assert call(ok, rows=-1) == L.EINVAL
    assert call(_t4(16, 32)) == L.EINVAL                           # other sizes
    assert call(_t4(16, 48, fmt=2)) == L.EUNSUPPORTED
    assert call(_t4(16, 48, ld=8)) == L.EINVAL                     # rows too short
    assert call(_t4(16, 48, ld=40)) == L.EINVAL                    # not 16-byte rows
    assert call(_t4(16, 48, codes=0x10008)) == L.EINVAL            # misaligned
    assert call(_t4(16, 48, scales=None)) == L.EINVAL
    assert call(_t4(16, 48, inv_scale=None)) == L.EINVAL           # NVFP4 has an inverse scale
    assert call(_t4(16, 48, inv_scale=0x50000)) == L.EINVAL        # of another state
    assert call(ok, st=None) == L.EINVAL
    assert call(ok, st=_state(fmt=1)) == L.EUNSUPPORTED            # e5m2 state
    assert call(ok, st=_state(eps=0.0)) == L.EINVAL
    assert call(ok, _t4(16, 48)) == L.EINVAL                       # not the transpose
    assert call(ok, _t4(48, 16, fmt=1, inv_scale=0x30000)) == L.EINVAL
    assert call(_t4(16, 48, fmt=1)) == L.EINVAL                    # MXFP4 takes no state
    assert call(_t4(16, 48, fmt=1, inv_scale=0x30000), st=None) == L.EINVAL


def test_product_refusals(lib):
    import quantised_gemm_gb300._lib as L
    p, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    nb = lib.fp8lin_workspace_bytes(0, 0, 0)

    def call(a, b, d=p, ldd=32, w=ws, n=nb):
        return lib.fp8lin_fp4_gemm(ctypes.byref(a), ctypes.byref(b), d, ldd, w, n, None)

    a, b = _t4(16, 48), _t4(32, 48)
    assert call(a, _t4(32, 64)) == L.EINVAL                        # K differs
    assert call(a, _t4(32, 48, fmt=1)) == L.EINVAL                 # formats differ
    assert call(a, b, d=None) == L.EINVAL
    assert call(a, b, d=ctypes.c_void_p(0x100001)) == L.EINVAL
    assert call(a, b, ldd=31) == L.EINVAL
    assert call(a, b, w=None) == L.EINVAL
    assert call(a, b, n=16) == L.EINVAL
    assert lib.fp8lin_fp4_dequantise(ctypes.byref(a), None, 48, 0, None) == L.EINVAL
    assert lib.fp8lin_fp4_dequantise(ctypes.byref(a), p, 47, 0, None) == L.EINVAL
    assert lib.fp8lin_fp4_dequantise(ctypes.byref(a), ctypes.c_void_p(0x100002), 48, 1,
                                     None) == L.EINVAL


def test_gradient_refusals(lib):
    import quantised_gemm_gb300._lib as L
    ws, norm = ctypes.c_void_p(0x200000), ctypes.c_void_p(0x300000)
    nb = lib.fp8lin_workspace_bytes(0, 0, 0)

    def grad(**kw):
        a = (L.GradC * 1)()
        a[0].g, a[0].out, a[0].n, a[0].g_f32, a[0].out_f32 = 0x1000, 0x2000, 8, 1, 1
        for k, v in kw.items():
            setattr(a[0], k, v)
        return a

    def call(a, count=1, max_norm=1.0, eps=1e-6, n=norm, w=ws):
        return lib.fp8lin_grad_clip_norm(a, count, max_norm, eps, n, w, nb, None)

    assert call(grad(), count=-1) == L.EINVAL
    assert call(None) == L.EINVAL
    assert call(grad(n=-1)) == L.EINVAL
    assert call(grad(g=None)) == L.EINVAL
    assert call(grad(out=None)) == L.EINVAL
    assert call(grad(g=0x1002)) == L.EINVAL                        # fp32 at 2 bytes
    assert call(grad(g_f32=0, g=0x1001)) == L.EINVAL
    assert call(grad(out=0x1000, out_f32=0)) == L.EINVAL           # in place with another type
    assert call(grad(), max_norm=-1.0) == L.EINVAL
    assert call(grad(), max_norm=float("nan")) == L.EINVAL
    assert call(grad(), eps=-1.0) == L.EINVAL
    assert call(grad(), n=None) == L.EINVAL
    assert call(grad(), n=ctypes.c_void_p(0x300002)) == L.EINVAL
    assert call(grad(), w=None) == L.EINVAL
    assert lib.fp8lin_grad_norm(grad(), 1, norm, None, nb, None) == L.EINVAL
    assert lib.fp8lin_grad_clip(grad(), 1, None, 1.0, 1e-6, None) == L.EINVAL


def test_own_inverse_scale_refusals(lib):
    import quantised_gemm_gb300._lib as L
    p, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    nb = lib.fp8lin_workspace_bytes(0, 0, 0)
    b = _t4(32, 48)
    for bad in (_t4(16, 48, own_inv=0x50002), _t4(16, 48, fmt=1, own_inv=0x50000)):
        b.fmt, b.inv_scale = bad.fmt, bad.inv_scale
        assert lib.fp8lin_fp4_dequantise(ctypes.byref(bad), p, 48, 0, None) == L.EINVAL
        assert lib.fp8lin_fp4_gemm(ctypes.byref(bad), ctypes.byref(b), p, 32, ws, nb, None) == L.EINVAL
        st = None if bad.fmt else ctypes.byref(_state())
        assert lib.fp8lin_fp4_quantise(p, 16, 48, 48, st, ctypes.byref(bad), None, ws, None) == L.EINVAL
