"""Limits of the token operators' calls, on the host (nothing is launched)."""
import ctypes as C
import os

import pytest

from differentiable_rasterization_amd import raster
from test_tokens_abi import BAD, P, _at_cfg, _docs, _h


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(raster.LIB_PATH):
        from differentiable_rasterization_amd import build
        build.build()
    return raster.load()


def test_searched_documents_are_bounded(lib):
    """Calls that search the documents take 2^20 of them; those that do not
    go on to their next check (here: an array is missing)."""
    many, rows = 1 << 21, 1 << 22
    c, h, s = _at_cfg(), C.byref(_h()), raster.gs_scan_config(1, 1, 64)

    def error(status):
        assert status == BAD
        return lib.gs_last_error().decode()
    for count, max_q_len, refused in ((many, 0, True), (many, 17, True), (many, 16, False),
                                      (1 << 20, 0, False)):
        d = C.byref(_docs(count=count, max_q_len=max_q_len))
        text = error(lib.gs_attention_fwd(C.byref(c), d, rows, rows, h, h, h, None, None, P,
                                          1 << 50, None))
        assert ("2^20" in text) == refused, text
    for count, max_q_len, saved, refused in ((many, 0, None, True), (many, 65, None, True),
                                             (many, 64, None, False), (many, 64, P, True),
                                             (1 << 20, 0, P, False)):
        d = C.byref(_docs(count=count, max_q_len=max_q_len))
        text = error(lib.gs_gated_scan_fwd(C.byref(s), d, rows, None, None, None, None, None,
                                           saved, P, 1 << 50, None))
        assert ("2^20" in text) == refused, text
    for count, size in ((many, False), (1 << 20, True)):
        d = C.byref(_docs(count=count, max_q_len=1))
        assert bool(lib.gs_attention_bwd_workspace_size(C.byref(c), d, rows, rows)) == size
        assert bool(lib.gs_gated_scan_saved_size(C.byref(s), d, rows)) == size
        assert ("2^20" in error(lib.gs_attention_bwd(C.byref(c), d, rows, rows, h, h, h, h, P, h, h,
                                                     h, None, P, 1 << 50, None))) != size
        assert ("2^20" in error(lib.gs_gated_scan_bwd(C.byref(s), d, rows, None, None, P, None, None,
                                                      None, None, None, P, 1 << 50, None))) != size


@pytest.mark.parametrize("softcap", [1e-40, 2.0 ** -101, 2.0 ** 101, 3e38])
def test_caps_beyond_fp32_products_are_refused(lib, softcap):
    c, d, h = _at_cfg(softcap=softcap), _docs(), C.byref(_h())
    assert lib.gs_attention_fwd(C.byref(c), C.byref(d), 8, 8, h, h, h, C.byref(_h(2 * P)), P, P,
                                1 << 40, None) == BAD
    assert lib.gs_attention_bwd_workspace_size(C.byref(c), C.byref(d), 8, 8) == 0
    for fine in (2.0 ** -100, 2.0 ** 100):
        c = _at_cfg(softcap=fine)
        assert lib.gs_attention_bwd_workspace_size(C.byref(c), C.byref(d), 8, 8) > 0
