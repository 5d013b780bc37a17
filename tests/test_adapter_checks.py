"""Argument checks of the adapters' C entry points: refused before anything touches a device."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from quantised_gemm_gb300 import build as qb
    qb.build()
    import quantised_gemm_gb300 as q
    return q.library()


P, Q = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)  # never dereferenced
ODD, HALF = ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)


def bank(**change):
    import quantised_gemm_gb300._lib as L
    c = L.AdaptersC(0x10000, 0x10000, 0x10000, 2, 64, 48, 8)
    for name, value in change.items():
        setattr(c, name, value)
    return c


def forward(lib, ad=None, **change):
    a = dict(x=P, ldx=64, index=P, route=None, rows=4, base=P, ldbase=48, y=Q, ldy=48, h=P, ws=P, nbytes=1 << 24)
    a.update(change)
    return lib.fp8lin_adapter_linear(None if ad == "null" else ctypes.byref(ad or bank()), a["x"], a["ldx"], a["index"],
                                     a["route"], a["rows"], a["base"], a["ldbase"], a["y"], a["ldy"], a["h"], a["ws"],
                                     a["nbytes"], None)


def backward(lib, ad=None, **change):
    a = dict(dy=P, lddy=48, x=P, ldx=64, h=P, index=P, route=None, rows=4, base=P, ldbase=64, dx=Q, lddx=64, dh=P, da=P,
             db=P, ws=P, nbytes=1 << 24)
    a.update(change)
    return lib.fp8lin_adapter_backward(ctypes.byref(ad or bank()), a["dy"], a["lddy"], a["x"], a["ldx"], a["h"], a["index"],
                                       a["route"], a["rows"], a["base"], a["ldbase"], a["dx"], a["lddx"], a["dh"], a["da"],
                                       a["db"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("call", [forward, backward])
def test_banks(lib, call):
    import quantised_gemm_gb300._lib as L
    for change in (dict(a=None), dict(a=0x10001), dict(b=None), dict(b=0x10001), dict(scale=None), dict(scale=0x10002),
                   dict(count=0), dict(k=0), dict(n=0), dict(rank=0), dict(count=-1), dict(rank=-1)):
        assert call(lib, bank(**change)) == L.EINVAL, change
    for change in (dict(count=1025), dict(rank=129), dict(k=(1 << 22) + 1), dict(n=(1 << 22) + 1)):
        assert call(lib, bank(**change)) == L.EUNSUPPORTED, change
    assert call(lib, rows=(1 << 24) + 1) == L.EUNSUPPORTED
    for change in (dict(rows=-1), dict(index=None), dict(index=HALF), dict(route=HALF), dict(ws=None), dict(ws=HALF),
                   dict(nbytes=100)):
        assert call(lib, **change) == L.EINVAL, change


def test_forward_refusals(lib):
    import quantised_gemm_gb300._lib as L
    assert forward(lib, "null") == L.EINVAL
    for change in (dict(x=None), dict(x=ODD), dict(ldx=63), dict(base=ODD), dict(ldbase=47), dict(y=None), dict(y=ODD),
                   dict(ldy=47), dict(y=P, ldy=56), dict(h=None), dict(h=HALF)):
        assert forward(lib, **change) == L.EINVAL, change


def test_backward_refusals(lib):
    import quantised_gemm_gb300._lib as L
    for change in (dict(dy=None), dict(dy=ODD), dict(lddy=47), dict(x=None), dict(ldx=63), dict(h=None), dict(h=HALF),
                   dict(base=ODD), dict(ldbase=63), dict(dx=ODD), dict(lddx=63), dict(dx=P, lddx=72), dict(dh=None),
                   dict(dh=HALF), dict(da=ODD), dict(db=ODD)):
        assert backward(lib, **change) == L.EINVAL, change


def test_route_refusals(lib):
    import quantised_gemm_gb300._lib as L
    assert lib.fp8lin_adapter_route_bytes(10, 3) >= 60
    for rows, count in ((-1, 3), (10, 0), (10, 1025), ((1 << 24) + 1, 3)):
        assert lib.fp8lin_adapter_route_bytes(rows, count) == 0
    assert lib.fp8lin_adapter_route(P, -1, 3, P, None) == L.EINVAL
    assert lib.fp8lin_adapter_route(P, 10, 0, P, None) == L.EINVAL
    assert lib.fp8lin_adapter_route(P, 10, 1025, P, None) == L.EUNSUPPORTED
    assert lib.fp8lin_adapter_route(P, (1 << 24) + 1, 3, P, None) == L.EUNSUPPORTED
    for index, route in ((None, P), (HALF, P), (P, None), (P, HALF)):
        assert lib.fp8lin_adapter_route(index, 10, 3, route, None) == L.EINVAL


def test_outputs_over_what_is_still_read(lib):
    import quantised_gemm_gb300._lib as L
    square = bank(k=48)
    R = ctypes.c_void_p(0x30000)
    assert forward(lib, square, y=P, base=Q, ldx=48) == L.EINVAL  # y is x
    for change in (dict(dx=P, dy=P, x=R), dict(dx=R, x=R)):
        assert backward(lib, square, base=Q, **change) == L.EINVAL, change
