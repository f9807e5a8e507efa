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
    # a few short rows are brought to 8 bits on the way
    assert size() == 0
    n = size(rows=40)
    assert n >= 40 * 64 + 40 * 4
    for bad in (dict(space=None), dict(space=5 * P + 16), dict(n=n - 1)):
        assert call(rows=40, **bad) == BAD
    assert call(rows=0, x=None, w=None, ws=None, y=None, space=None, n=0) == OK


def _h(data=P, row=1024, head=64):
    return raster.gs_heads(data, row, head)


def _docs(**kw):
    a = dict(count=2, max_q_len=0, max_k_len=0, q_start=P, q_len=P, k_start=P, k_len=P,
             prefix=None)
    a.update(kw)
    return raster.gs_documents(*[a[n] for n, _ in raster.gs_documents._fields_])


def _c(first=16, **kw):
    """A cache of 8 rows, 2 heads of 64 in 8 bits."""
    a = dict(codes=first * P, low=(first + 1) * P, step=(first + 2) * P, row=128, head=64, ld=8,
             bits=8)
    a.update(kw)
    return raster.gs_codes(*[a[n] for n, _ in raster.gs_codes._fields_])


BAD_CACHES = [dict(codes=None), dict(low=None), dict(step=None), dict(codes=16 * P + 8),
              dict(low=17 * P + 2), dict(step=18 * P + 1), dict(row=126), dict(head=62),
              dict(row=64), dict(head=32), dict(row=1 << 25), dict(head=-64), dict(row=-128),
              dict(ld=7), dict(ld=1 << 41), dict(bits=2), dict(bits=0), dict(bits=16),
              dict(low=18 * P), dict(low=16 * P), dict(head=0)]
BAD_DOCS = [dict(count=-1), dict(count=1 << 25), dict(count=(1 << 20) + 1), dict(max_q_len=-1),
            dict(max_k_len=-5), dict(q_start=None), dict(q_len=None), dict(k_start=None),
            dict(k_len=None)]


def _cache_cfg(dtype=1, heads=2, dim=64):
    return raster.gs_cache_config(dtype, heads, dim)


def _write(lib, c=_cache_cfg(), d=_docs(), rq=8, rk=8, k=_h(), v=_h(2 * P), kc=_c(), vc=_c(24)):
    return lib.gs_cache_write(_b(c), _b(d), rq, rk, _b(k), _b(v), _b(kc), _b(vc), None)


def _read(lib, c=_cache_cfg(), d=_docs(), rq=8, rk=8, k=_h(), v=_h(2 * P), kc=_c(), vc=_c(24)):
    return lib.gs_cache_read(_b(c), _b(d), rq, rk, _b(kc), _b(vc), _b(k), _b(v), None)


@pytest.mark.parametrize("call", [_write, _read])
def test_cache_calls_are_checked(lib, call):
    for bad in (dict(dtype=3), dict(dtype=-1), dict(heads=0), dict(heads=65537), dict(dim=0),
                dict(dim=8), dict(dim=72), dict(dim=144)):
        assert call(lib, _cache_cfg(**bad)) == BAD
    assert lib.gs_last_error().decode()
    assert call(lib, None) == BAD and call(lib, d=None) == BAD
    for bad in BAD_DOCS:
        assert call(lib, d=_docs(**bad)) == BAD
    for rows in (-1, 1 << 31, 1 << 30):
        assert call(lib, rq=rows) == BAD and call(lib, rk=rows) == BAD
    for bad in BAD_CACHES:
        assert call(lib, kc=_c(**bad)) == BAD
    assert call(lib, kc=None) == BAD and call(lib, vc=None) == BAD
    assert call(lib, vc=_c(24, bits=4)) == BAD                   # other bits
    for t in (None, _h(None), _h(P + 8), _h(row=1020), _h(head=-64)):
        assert call(lib, k=t) == BAD and call(lib, v=t) == BAD
    for at in (16, 17, 18, 24, 25, 26):                          # a cache over the tokens
        assert call(lib, k=_h(at * P)) == BAD and call(lib, v=_h(at * P)) == BAD
    none = _docs(count=0, q_start=None, q_len=None, k_start=None, k_len=None)
    assert call(lib, d=none, rq=0, rk=0, k=None, v=None) == OK
    assert call(lib, rq=0, k=None, v=None) == OK


def test_caches_that_are_written_are_apart(lib):
    assert _write(lib, vc=_c()) == BAD
    assert _write(lib, vc=_c(24, low=17 * P)) == BAD and _write(lib, vc=_c(24, step=16 * P)) == BAD
    assert _write(lib, rk=0, kc=_c(codes=None, low=None, step=None), vc=_c(24)) == OK
    assert _read(lib, k=_h(row=32)) == BAD and _read(lib, v=_h(2 * P, head=0)) == BAD
    assert _read(lib, v=_h()) == BAD


def _at_cfg(**kw):
    a = dict(dtype=1, heads_q=4, heads_k=2, head_dim=64, causal=1, scale=0.1, softcap=0.0,
             slopes=None)
    a.update(kw)
    return raster.gs_attention_config(*[a[n] for n, _ in raster.gs_attention_config._fields_])


def _attend(lib, c=_at_cfg(), d=_docs(), shared=None, rq=8, rk=8, q=_h(), kc=_c(), vc=_c(24),
            out=_h(2 * P), lse=3 * P, space=P, n=1 << 40):
    return lib.gs_cached_attention_fwd(_b(c), _b(d), _b(shared), rq, rk, _b(q), _b(kc), _b(vc),
                                       _b(out), lse, space, n, None)


def _size(lib, c=_at_cfg(), bits=8, d=_docs(), shared=None, rq=8, rk=1 << 20):
    return lib.gs_cached_attention_fwd_workspace_size(_b(c), bits, _b(d), _b(shared), rq, rk)


def test_attention_over_caches_is_checked(lib):
    for bad in (dict(dtype=0), dict(dtype=3), dict(heads_q=0), dict(heads_k=0), dict(heads_k=3),
                dict(head_dim=72), dict(head_dim=144), dict(head_dim=0), dict(causal=2),
                dict(scale=float("nan")), dict(softcap=-1.0), dict(softcap=float("inf"))):
        assert _attend(lib, _at_cfg(**bad)) == BAD and _size(lib, _at_cfg(**bad)) == 0
    assert _attend(lib, None) == BAD and _size(lib, None) == 0
    for bits in (0, 2, 16, -8):
        assert _size(lib, bits=bits) == 0
    for bad in BAD_DOCS:
        assert _attend(lib, d=_docs(**bad)) == BAD and _size(lib, d=_docs(**bad)) == 0
        assert _attend(lib, shared=_docs(**bad)) == BAD and _size(lib, shared=_docs(**bad)) == 0
    assert _attend(lib, d=None) == BAD
    own_rows = _docs(k_start=None, k_len=None)
    assert _attend(lib, shared=own_rows) == BAD                  # shared keys need ranges
    assert _attend(lib, _at_cfg(slopes=P), shared=_docs()) == BAD
    for rows in (-1, 1 << 31, 1 << 30):
        assert _attend(lib, rq=rows) == BAD and _attend(lib, rk=rows) == BAD
    for bad in BAD_CACHES:
        assert _attend(lib, kc=_c(**bad)) == BAD and _attend(lib, vc=_c(**bad)) == BAD
    assert _attend(lib, kc=None) == BAD and _attend(lib, vc=None) == BAD
    assert _attend(lib, vc=_c(24, bits=4)) == BAD
    assert _attend(lib, q=None) == BAD and _attend(lib, q=_h(P + 8)) == BAD
    assert _attend(lib, out=_h()) == BAD and _attend(lib, out=_h(2 * P, row=64)) == BAD
    for at in (16, 17, 18, 24, 25, 26):
        assert _attend(lib, out=_h(at * P)) == BAD
    assert _attend(lib, lse=3 * P + 2) == BAD
    none = _docs(count=0, q_start=None, q_len=None, k_start=None, k_len=None)
    assert _attend(lib, d=none, q=None, out=None, space=None, n=0) == OK
    assert _attend(lib, rq=0, q=None, out=None, space=None, n=0) == OK


def test_attention_over_caches_needs_its_workspace(lib):
    n = _size(lib)
    assert n > 0 and _size(lib, shared=_docs()) > n
    big = _c(ld=1 << 20), _c(24, ld=1 << 20)
    call = lambda **kw: _attend(lib, rk=1 << 20, kc=big[0], vc=big[1], **kw)
    assert call(space=None, n=n) == BAD and call(space=P + 16, n=n) == BAD and call(n=n - 1) == BAD
