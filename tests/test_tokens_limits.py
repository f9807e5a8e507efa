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


def _qk_call(lib, q, k, oq, ok, back=None):
    """Status of a call of 8 tokens, 4 and 2 heads of 64; a workspace that is
    too small, or a weight that is missing, ends the ones that pass."""
    b = C.byref
    c = raster.gs_qk_config(1, 4, 2, 64, 0, 0, 0 if back is None else 1, 1e-6, 1.0)
    if back is None:
        return lib.gs_qk_norm_rope_fwd(b(c), 8, None, None, None, None, b(q), b(k), b(oq), b(ok),
                                       None), ""
    status = lib.gs_qk_norm_rope_bwd(b(c), 8, None, None, P, P, b(q), b(k), b(back[0]),
                                     b(back[1]), b(oq), b(ok), P, P, P, 1, None)
    return status, lib.gs_last_error().decode()


def test_outputs_over_other_elements_are_refused(lib):
    """An output at an input's address with other strides writes tokens that
    are still to be read."""
    q, k, o, p = _h(P), _h(2 * P), _h(3 * P), _h(4 * P)
    other = lambda n: _h(n * P, row=256)
    assert _qk_call(lib, q, k, other(1), p)[0] == BAD
    assert _qk_call(lib, q, k, o, other(2))[0] == BAD
    assert _qk_call(lib, q, k, k, p)[0] == BAD and _qk_call(lib, q, k, o, q)[0] == BAD
    assert _qk_call(lib, q, k, o, _h(3 * P, row=512))[0] == BAD
    dq, dk = _h(5 * P), _h(6 * P)
    fine = "workspace smaller"
    for a, b in ((o, p), (dq, dk), (q, k), (_h(7 * P, row=512), _h(8 * P, row=128))):
        assert fine in _qk_call(lib, q, k, a, b, (dq, dk))[1]
    for a, b in ((other(5), p), (o, other(6)), (other(1), p), (o, other(2)), (dk, p), (o, dq),
                 (k, p), (o, q), (o, o)):
        status, text = _qk_call(lib, q, k, a, b, (dq, dk))
        assert status == BAD and fine not in text, text
