"""Refusals of the calls of serving in 8 and 4 bits, on the host, before anything
is launched (no GPU is touched)."""
import ctypes as C
import os

import pytest

from differentiable_rasterization_amd import raster

BAD, OK = raster.GS_ERR_INVALID_ARGUMENT, raster.GS_OK
P = 4096  # never dereferenced: validation fails first, or nothing is launched


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(raster.LIB_PATH):
        from differentiable_rasterization_amd import build
        build.build()
    return raster.load()


def _r(data=P, row=1024):
    return raster.gs_rows(data, row)


def _b(x):
    return None if x is None else C.byref(x)


def test_rows_to_8_bits_are_checked(lib):
    def call(dtype=1, rows=4, channels=64, x=_r(), codes=2 * P, scales=3 * P):
        return lib.gs_quantize_rows(dtype, rows, channels, _b(x), codes, scales, None)
    assert call(dtype=3) == BAD and call(dtype=-1) == BAD
    assert lib.gs_last_error().decode()
    assert call(rows=-1) == BAD and call(rows=1 << 31) == BAD
    for channels in (0, 8, 24, -16, 131072):
        assert call(channels=channels) == BAD
    assert call(x=None) == BAD and call(x=_r(None)) == BAD and call(x=_r(P + 2)) == BAD
    assert call(x=_r(row=1020)) == BAD and call(x=_r(row=1 << 29)) == BAD
    assert call(codes=None) == BAD and call(codes=2 * P + 8) == BAD and call(codes=P) == BAD
    assert call(scales=None) == BAD and call(scales=P + 2) == BAD and call(scales=P) == BAD
    assert call(rows=0, x=None, codes=None, scales=None) == OK


def test_products_are_checked(lib):
    def cfg(dtype=1, inputs=64, outputs=32):
        return raster.gs_linear_config(dtype, inputs, outputs)

    def call(c=cfg(), rows=4, x=_r(), w=2 * P, ws=3 * P, bias=None, y=_r(4 * P), space=5 * P,
             n=1 << 40):
        return lib.gs_linear_i8(_b(c), rows, _b(x), w, ws, bias, _b(y), space, n, None)

    def size(c=cfg(), rows=4):
        return lib.gs_linear_i8_workspace_size(_b(c), rows)
    for bad in (dict(dtype=3), dict(dtype=-1), dict(inputs=0), dict(inputs=24),
                dict(inputs=131072), dict(outputs=0), dict(outputs=12), dict(outputs=1 << 25)):
        assert call(cfg(**bad)) == BAD and size(cfg(**bad)) == 0
    assert call(None) == BAD and size(None) == 0
    for rows in (-1, 1 << 31):
        assert call(rows=rows) == BAD and size(rows=rows) == 0
    big = cfg(outputs=1 << 24)
    assert call(big, rows=(1 << 13) + 1, y=_r(4 * P, 1 << 24)) == BAD
    assert size(big, (1 << 13) + 1) == 0 and size(big, 1 << 13) > 0
    assert call(x=None) == BAD and call(x=_r(None)) == BAD and call(x=_r(P + 8)) == BAD
    assert call(w=None) == BAD and call(w=2 * P + 4) == BAD
    assert call(ws=None) == BAD and call(ws=3 * P + 2) == BAD and call(bias=3 * P + 1) == BAD
    assert call(y=None) == BAD and call(y=_r(4 * P, 24)) == BAD       # rows overlap
    for alias in (P, 2 * P, 3 * P):
        assert call(y=_r(alias)) == BAD
    assert call(bias=4 * P) == BAD
    n = size()
    assert n >= 4 * 64 + 4 * 4
    assert call(space=None) == BAD and call(space=5 * P + 16) == BAD and call(n=n - 1) == BAD
    assert call(rows=0, x=None, w=None, ws=None, y=None, space=None, n=0) == OK
