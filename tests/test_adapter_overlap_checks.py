"""Buffers of the adapters' backward that overlap: refused before anything touches a device."""
import ctypes

import pytest

from test_adapter_checks import backward, bank, lib  # noqa: F401


@pytest.mark.parametrize("apart", [0, 4, 124, -4, -124])
def test_dh_over_the_h_that_db_needs(lib, apart):  # noqa: F811
    """4 rows of rank 8 are 128 bytes.  dh is written first: dB would be made of it instead of h."""
    import quantised_gemm_gb300._lib as L
    x, dx = ctypes.c_void_p(0x30000), ctypes.c_void_p(0x40000)
    h, dh = ctypes.c_void_p(0x50000), ctypes.c_void_p(0x50000 + apart)
    assert backward(lib, bank(), x=x, dx=dx, h=h, dh=dh) == L.EINVAL
