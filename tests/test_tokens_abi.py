"""Refusals of the token operators' calls, on the host, before anything is
launched (no GPU is touched)."""
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


def _h(data=P, row=1024, head=64):
    return raster.gs_heads(data, row, head)


def _docs(**kw):
    a = dict(count=2, max_q_len=0, max_k_len=0, q_start=P, q_len=P, k_start=None, k_len=None,
             prefix=None)
    a.update(kw)
    return raster.gs_documents(*[a[n] for n, _ in raster.gs_documents._fields_])


def _qk_cfg(**kw):
    a = dict(dtype=1, heads_q=4, heads_k=2, head_dim=64, rotary_dim=64, interleaved=0, norm=1,
             eps=1e-6, amplitude=1.0)
    a.update(kw)
    return raster.gs_qk_config(*[a[n] for n, _ in raster.gs_qk_config._fields_])


BAD_QK = [dict(dtype=3), dict(dtype=-1), dict(heads_q=0), dict(heads_k=0), dict(head_dim=60),
          dict(head_dim=0), dict(head_dim=520), dict(rotary_dim=24), dict(rotary_dim=80),
          dict(rotary_dim=-16), dict(interleaved=2), dict(norm=-1), dict(eps=-1.0),
          dict(eps=float("nan")), dict(amplitude=float("inf"))]


@pytest.mark.parametrize("kw", BAD_QK)
def test_qk_config_is_checked(lib, kw):
    h = C.byref(_h())
    c = _qk_cfg(**kw)
    assert lib.gs_qk_norm_rope_fwd(C.byref(c), 8, P, P, P, P, h, h, h, h, None) == BAD
    assert lib.gs_last_error().decode()
    assert lib.gs_qk_norm_rope_bwd_workspace_size(C.byref(c), 8) == 0
    assert lib.gs_qk_norm_rope_bwd(C.byref(c), 8, P, P, P, P, h, h, h, h, h, h, P, P, P, 1 << 30,
                                   None) == BAD


def test_qk_arrays_are_checked(lib):
    c, h = _qk_cfg(), _h()

    def fwd(cfg=c, rows=8, pos=P, freq=P, wq=P, wk=P, q=h, k=h, oq=h, ok=h):
        b = lambda x: None if x is None else C.byref(x)
        return lib.gs_qk_norm_rope_fwd(C.byref(cfg), rows, pos, freq, wq, wk, b(q), b(k), b(oq),
                                       b(ok), None)
    assert lib.gs_qk_norm_rope_fwd(None, 8, P, P, P, P, *[C.byref(h)] * 4, None) == BAD
    assert fwd(rows=-1) == BAD
    assert fwd(rows=1 << 31) == BAD
    assert fwd(rows=1 << 29) == BAD                    # rows times heads
    assert fwd(pos=None) == BAD and fwd(freq=None) == BAD
    assert fwd(wq=None) == BAD and fwd(wk=P + 4) == BAD
    assert fwd(q=None) == BAD and fwd(k=_h(None)) == BAD
    assert fwd(q=_h(P + 2)) == BAD                     # misaligned
    assert fwd(q=_h(row=1020)) == BAD and fwd(k=_h(head=-64)) == BAD
    assert fwd(q=_h(row=1 << 29)) == BAD
    assert fwd(oq=_h(row=64)) == BAD                   # rows overlap
    assert fwd(ok=_h(head=0)) == BAD                   # heads overlap
    assert fwd(rows=0, pos=None, q=None, k=None, oq=None, ok=None) == OK
    n = lib.gs_qk_norm_rope_bwd_workspace_size(C.byref(c), 8)
    assert n > 0 and lib.gs_qk_norm_rope_bwd_workspace_size(C.byref(c), -1) == 0

    def bwd(ws=P, nb=n, dwq=P, dq=h):
        b = C.byref(h)
        return lib.gs_qk_norm_rope_bwd(C.byref(c), 8, P, P, P, P, b, b, b, b, C.byref(dq), b, dwq,
                                       P, ws, nb, None)
    assert bwd(ws=None) == BAD and bwd(ws=P + 16) == BAD and bwd(nb=n - 1) == BAD
    assert bwd(dwq=None) == BAD and bwd(dq=_h(row=0)) == BAD


def _at_cfg(**kw):
    a = dict(dtype=1, heads_q=4, heads_k=2, head_dim=64, causal=1, scale=0.1, softcap=0.0,
             slopes=None)
    a.update(kw)
    return raster.gs_attention_config(*[a[n] for n, _ in raster.gs_attention_config._fields_])


BAD_AT = [dict(dtype=0), dict(dtype=3), dict(heads_q=0), dict(heads_k=0), dict(heads_k=3),
          dict(heads_q=2, heads_k=4), dict(head_dim=136), dict(head_dim=0), dict(head_dim=20),
          dict(causal=2), dict(scale=float("nan")), dict(scale=float("inf")),
          dict(softcap=-1.0), dict(softcap=float("inf"))]


@pytest.mark.parametrize("kw", BAD_AT)
def test_attention_config_is_checked(lib, kw):
    c, d, h = _at_cfg(**kw), _docs(), C.byref(_h())
    assert lib.gs_attention_fwd(C.byref(c), C.byref(d), 8, 8, h, h, h, C.byref(_h(2 * P)), P, P,
                                1 << 40, None) == BAD
    assert lib.gs_last_error().decode()
    assert lib.gs_attention_fwd_workspace_size(C.byref(c), C.byref(d), 8, 8) == 0
    assert lib.gs_attention_bwd_workspace_size(C.byref(c), C.byref(d), 8, 8) == 0


@pytest.mark.parametrize("kw", [dict(count=-1), dict(count=1 << 25), dict(max_q_len=-1),
                                dict(max_k_len=-5), dict(q_start=None), dict(q_len=None),
                                dict(k_start=P), dict(k_len=P)])
def test_documents_are_checked(lib, kw):
    d, h = _docs(**kw), C.byref(_h())
    assert lib.gs_attention_fwd(C.byref(_at_cfg()), C.byref(d), 8, 8, h, h, h,
                                C.byref(_h(2 * P)), P, P, 1 << 40, None) == BAD
    if "k_start" in kw or "k_len" in kw:
        return
    s = raster.gs_scan_config(1, 1, 64)
    r = raster.gs_rows(P, 64)
    assert lib.gs_gated_scan_fwd(C.byref(s), C.byref(d), 8, C.byref(r), C.byref(r), None,
                                 C.byref(raster.gs_rows(2 * P, 64)), None, None, P, 1 << 40,
                                 None) == BAD


def test_attention_arrays_are_checked(lib):
    c, d = _at_cfg(), _docs()
    b = lambda x: None if x is None else C.byref(x)

    def fwd(docs=d, rq=8, rk=8, q=_h(), k=_h(), v=_h(), o=_h(2 * P)):
        return lib.gs_attention_fwd(C.byref(c), b(docs), rq, rk, b(q), b(k), b(v), b(o), None, P,
                                    1 << 40, None)
    assert fwd(docs=None) == BAD
    assert fwd(rq=-1) == BAD and fwd(rk=1 << 31) == BAD and fwd(rq=1 << 30) == BAD
    assert fwd(q=None) == BAD and fwd(k=None) == BAD and fwd(v=_h(None)) == BAD
    assert fwd(o=_h()) == BAD                          # aliases an input
    assert fwd(o=_h(2 * P, row=64)) == BAD             # overlapping output
    assert fwd(k=_h(P + 8)) == BAD and fwd(v=_h(row=1 << 30)) == BAD
    assert fwd(docs=_docs(count=0, q_start=None, q_len=None)) == OK
    assert fwd(rq=0, q=None, o=None) == OK
    n = lib.gs_attention_bwd_workspace_size(C.byref(c), C.byref(d), 8, 8)
    assert n > 0

    def bwd(lse=P, do=_h(), dq=_h(2 * P), dk=_h(3 * P), dv=_h(4 * P), ws=P, nb=n):
        h = C.byref(_h())
        return lib.gs_attention_bwd(C.byref(c), C.byref(d), 8, 8, h, h, h, h, lse, b(do), b(dq),
                                    b(dk), b(dv), ws, nb, None)
    assert bwd(lse=None) == BAD and bwd(do=None) == BAD and bwd(dq=None) == BAD
    assert bwd(dk=_h(4 * P)) == BAD                    # dk and dv alias
    assert bwd(dv=_h(P)) == BAD and bwd(dq=_h(P)) == BAD
    assert bwd(ws=None) == BAD and bwd(ws=P + 64) == BAD and bwd(nb=n - 1) == BAD


def test_scan_arguments_are_checked(lib):
    d, r, out = _docs(), raster.gs_rows(P, 128), raster.gs_rows(2 * P, 128)

    def fwd(cfg=(1, 1, 64), docs=d, rows=1000, gate=r, x=r, y=out, h=None, ws=P, nb=1 << 40):
        c = raster.gs_scan_config(*cfg)
        b = lambda t: None if t is None else C.byref(t)
        return lib.gs_gated_scan_fwd(C.byref(c), b(docs), rows, b(gate), b(x), h, b(y), None, None,
                                     ws, nb, None)
    for cfg in ((3, 1, 64), (1, 2, 64), (1, 1, 0), (1, 1, 60), (1, 1, (1 << 24) + 8)):
        assert fwd(cfg=cfg) == BAD
        assert lib.gs_gated_scan_fwd_workspace_size(C.byref(raster.gs_scan_config(*cfg)),
                                                    C.byref(d), 1000) == 0
    assert fwd(rows=-1) == BAD and fwd(rows=1 << 31) == BAD
    assert fwd(cfg=(1, 1, 1 << 24), rows=1 << 30) == BAD   # a grid too large
    assert fwd(docs=None) == BAD
    assert fwd(gate=None) == BAD and fwd(x=raster.gs_rows(P + 4, 128)) == BAD
    assert fwd(x=raster.gs_rows(P, 100)) == BAD
    assert fwd(y=raster.gs_rows(2 * P, 32)) == BAD         # rows overlap
    assert fwd(y=r) == BAD                                 # aliases an input
    assert fwd(h=P + 4) == BAD
    assert fwd(ws=None) == BAD and fwd(nb=10) == BAD and fwd(ws=P + 8) == BAD
    assert fwd(docs=_docs(count=0)) == OK
    c = raster.gs_scan_config(1, 1, 64)
    # short documents need no workspace; what is saved is needed for any
    assert lib.gs_gated_scan_fwd_workspace_size(C.byref(c), C.byref(_docs(max_q_len=4)), 1000) == 0
    assert lib.gs_gated_scan_saved_size(C.byref(c), C.byref(d), 1000) > 0

    def bwd(saved=P, dy=r, df=out, dx=raster.gs_rows(3 * P, 128), ws=P, nb=1 << 40):
        b = C.byref
        return lib.gs_gated_scan_bwd(b(c), b(d), 1000, b(r), b(r), saved, b(dy), None, b(df),
                                     b(dx), None, ws, nb, None)
    assert bwd(saved=None) == BAD and bwd(df=r) == BAD and bwd(dx=out) == BAD
    assert bwd(ws=None) == BAD and bwd(nb=10) == BAD


def test_python_views_are_checked():
    import torch
    with pytest.raises(ValueError):
        raster.heads(torch.zeros(4, 4))
    with pytest.raises(ValueError):
        raster.heads(torch.zeros(4, 4, 8).transpose(1, 2))
    with pytest.raises(ValueError):
        raster.rows(torch.zeros(4, 8).T)
    with pytest.raises(ValueError):
        raster.documents(torch.zeros(3, dtype=torch.int64), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        raster.documents(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        raster.attention_config(torch.float64, 2, 2, 64, 0.1)
    with pytest.raises(ValueError):
        raster.attention_config(torch.float16, 2, 2, 64, 0.1, slopes=torch.zeros(3))
