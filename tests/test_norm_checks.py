"""Argument checks of the layer norm's C entry points: refused before anything touches a device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from quantised_gemm_gb300 import build as qb
    qb.build()
    import quantised_gemm_gb300 as q
    return q.library()


P = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10002)


def forward(lib, **change):
    a = dict(x=P, ldx=64, r=None, ldr=0, h=None, ldh=0, w=P, b=P, f32=0, rows=4, cols=64, eps=1e-5, y=P, ldy=64,
             stats=P, amax=None, ws=P)
    a.update(change)
    return lib.fp8lin_layer_norm(a["x"], a["ldx"], a["r"], a["ldr"], a["h"], a["ldh"], a["w"], a["b"], a["f32"],
                                 a["rows"], a["cols"], a["eps"], a["y"], a["ldy"], a["stats"], a["amax"], a["ws"], None)


def backward(lib, **change):
    a = dict(dy=P, lddy=64, x=P, ldx=64, w=P, f32=0, stats=P, rows=4, cols=64, dres=None, lddres=0, dx=P, lddx=64,
             dw=P, db=P, amax=None, ws=P, nbytes=1 << 24)
    a.update(change)
    return lib.fp8lin_layer_norm_backward(a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["f32"], a["stats"], a["rows"],
                                          a["cols"], a["dres"], a["lddres"], a["dx"], a["lddx"], a["dw"], a["db"],
                                          a["amax"], a["ws"], a["nbytes"], None)


def test_forward_refusals(lib):
    import quantised_gemm_gb300._lib as L
    for change in (dict(rows=-1), dict(cols=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(x=ODD),
                   dict(ldx=63), dict(y=None), dict(ldy=63), dict(w=None), dict(w=ODD), dict(f32=1, w=HALF), dict(b=ODD),
                   dict(stats=HALF), dict(amax=HALF), dict(amax=P, ws=None), dict(amax=P, ws=HALF), dict(r=P, ldr=64),
                   dict(h=P, ldh=64), dict(r=P, ldr=63, h=P, ldh=64), dict(r=P, ldr=64, h=ODD, ldh=64)):
        assert forward(lib, **change) == L.EINVAL, change
    assert forward(lib, cols=0) == L.EUNSUPPORTED
    assert forward(lib, cols=16385, ldx=1 << 20, ldy=1 << 20) == L.EUNSUPPORTED


def test_backward_refusals(lib):
    import quantised_gemm_gb300._lib as L
    for change in (dict(rows=-1), dict(cols=-1), dict(dy=None), dict(dy=ODD), dict(lddy=63), dict(x=None), dict(ldx=63),
                   dict(w=None), dict(f32=1, dw=HALF), dict(db=ODD), dict(stats=None), dict(stats=HALF), dict(dx=ODD),
                   dict(lddx=63), dict(dres=P, lddres=63), dict(amax=HALF), dict(amax=P, dx=None), dict(ws=None),
                   dict(ws=HALF), dict(nbytes=16384)):
        assert backward(lib, **change) == L.EINVAL, change
    assert backward(lib, cols=16385, lddy=1 << 20, ldx=1 << 20, lddx=1 << 20) == L.EUNSUPPORTED
    assert backward(lib, cols=0) == L.EUNSUPPORTED


def test_an_output_over_an_input_has_its_rows(lib):
    import quantised_gemm_gb300._lib as L
    Q = ctypes.c_void_p(0x20000)
    R = ctypes.c_void_p(0x30000)
    for change in (dict(ldy=72), dict(y=Q, r=Q, ldr=72, h=R, ldh=64), dict(y=Q, r=R, ldr=64, h=Q, ldh=72),
                   dict(y=Q, r=R, ldr=64, h=P, ldh=72), dict(y=Q, r=R, ldr=64, h=R, ldh=72)):
        assert forward(lib, **change) == L.EINVAL, change
    for change in (dict(lddx=72), dict(dx=Q, dres=Q, lddres=72)):
        assert backward(lib, **change) == L.EINVAL, change
