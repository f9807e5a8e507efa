"""The binding refuses arrays that a kernel would read or write past their
end: another type, too few elements, strides, host memory.  The library is
replaced by one that only counts calls, so nothing is launched."""
import types

import pytest
import torch

from differentiable_rasterization_amd import raster

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
NO_STREAM = types.SimpleNamespace(cuda_stream=0)


class CountingLibrary:
    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                return 1024
            self.calls += 1
            return raster.GS_OK
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = CountingLibrary()
    monkeypatch.setattr(raster, "_lib", lib)
    # host tensors stand in for device memory here
    monkeypatch.setattr(raster, "_on_device", lambda t: True, raising=False)
    return lib


def _t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


N, HQ, HK, D, C, DOCS = 6, 4, 2, 32, 16, 3


def _qk(norm=True, rotary=D):
    cfg = raster.qk_config(BF16, HQ, HK, D, rotary, norm=norm)
    q, k = _t(N, HQ, D), _t(N, HK, D)
    a = dict(positions=_t(N, dtype=I32), inv_freq=_t(D // 2, dtype=F32), wq=_t(D, dtype=F32),
             wk=_t(D, dtype=F32), q=q, k=k)
    fwd = dict(a, q_out=q, k_out=k)
    bwd = dict(a, dL_dq_out=q, dL_dk_out=k, dL_dq=q, dL_dk=k, dL_dwq=_t(D, dtype=F32),
               dL_dwk=_t(D, dtype=F32), workspace=_t(512, dtype=U8))
    return ((raster.gs_qk_norm_rope_fwd, (cfg, N), fwd, ()),
            (raster.gs_qk_norm_rope_bwd, (cfg, N), bwd, (512,)))


def _docs():
    return raster.documents(_t(DOCS, dtype=I32), _t(DOCS, dtype=I32))


def _attention():
    cfg = raster.attention_config(BF16, HQ, HK, D, 0.1)
    q, k = _t(N, HQ, D), _t(N + 3, HK, D)
    a = dict(q=q, k=k, v=k, out=q, lse=_t(HQ, N, dtype=F32))
    fwd = dict(a, workspace=_t(512, dtype=U8))
    bwd = dict(a, dL_dout=q, dL_dq=q, dL_dk=k, dL_dv=k, workspace=_t(512, dtype=U8))
    return ((raster.gs_attention_fwd, (cfg, _docs(), N, N + 3), fwd, (512,)),
            (raster.gs_attention_bwd, (cfg, _docs(), N, N + 3), bwd, (512,)))


def _scan():
    cfg = raster.scan_config(BF16, C)
    x, h = _t(N, C), _t(DOCS, C, dtype=F32)
    fwd = dict(gate=x, x=x, state_in=h, y=x, state_out=h, saved=_t(1024, dtype=U8),
               workspace=_t(512, dtype=U8))
    bwd = dict(gate=x, x=x, saved=_t(1024, dtype=U8), dL_dy=x, dL_dstate_out=h, dL_dgate=x,
               dL_dx=x, dL_dstate_in=h, workspace=_t(512, dtype=U8))
    return ((raster.gs_gated_scan_fwd, (cfg, _docs(), N), fwd, (512,)),
            (raster.gs_gated_scan_bwd, (cfg, _docs(), N), bwd, (512,)))


def _calls():
    return _qk() + _attention() + _scan()


QK = "positions inv_freq wq wk q k "
NAMES = [(i, name) for i, names in enumerate((
    QK + "q_out k_out",
    QK + "dL_dq_out dL_dk_out dL_dq dL_dk dL_dwq dL_dwk workspace",
    "q k v out lse workspace",
    "q k v out lse dL_dout dL_dq dL_dk dL_dv workspace",
    "gate x state_in y state_out saved workspace",
    "gate x saved dL_dy dL_dstate_out dL_dgate dL_dx dL_dstate_in workspace"))
    for name in names.split()]


def _call(i, **other):
    fn, first, arrays, last = _calls()[i]
    fn(*first, *dict(arrays, **other).values(), *last, stream=NO_STREAM)


@pytest.mark.parametrize("i,name", NAMES)
def test_arrays_that_do_not_fit_are_refused(lib, i, name):
    _call(i)
    assert lib.calls == 1
    assert list(_calls()[i][2]) == [n for j, n in NAMES if j == i]
    t = _calls()[i][2][name]
    bad = [t[:-1] if t.dim() == 1 else t[:-1].clone()]           # too few
    if t.dtype != U8:
        bad += [t.to(torch.float16), t.to(torch.float64)]        # another type
        bad.append(t[..., :-8].contiguous())                     # shorter rows
    if t.dim() < 3 and t.dtype != BF16:
        bad.append(torch.zeros_like(t[:1]).expand(t.shape))      # no memory behind it
    for b in bad:
        with pytest.raises(ValueError):
            _call(i, **{name: b})
    if t.dim() == 3:
        with pytest.raises(ValueError):
            _call(i, **{name: raster.heads(bad[0])})             # a view made before
        with pytest.raises(ValueError):
            _call(i, **{name: t[:, 1:]})                         # a head too few
    assert lib.calls == 1


@pytest.mark.parametrize("i,name", NAMES)
def test_host_memory_is_refused(lib, monkeypatch, i, name):
    fn, first, arrays, last = _calls()[i]
    host = arrays[name].clone()
    monkeypatch.setattr(raster, "_on_device", lambda t: t is not host)
    with pytest.raises(ValueError):
        fn(*first, *dict(arrays, **{name: host}).values(), *last, stream=NO_STREAM)
    assert lib.calls == 0


def test_host_documents_and_slopes_are_refused():
    with pytest.raises(ValueError):
        raster.documents(_t(3, dtype=I32), _t(3, dtype=I32))
    with pytest.raises(ValueError):
        raster.attention_config(BF16, 3, 3, D, 0.1, slopes=_t(3, dtype=F32))


def test_what_the_configuration_leaves_out_is_not_looked_at(lib):
    none = dict(positions=None, inv_freq=None, wq=None, wk=None)
    for (fn, first, arrays, last), (more) in zip(_qk(norm=False, rotary=0),
                                                 ({}, dict(dL_dwq=None, dL_dwk=None))):
        fn(*first, *dict(arrays, **none, **more).values(), *last, stream=NO_STREAM)
        fn(*first, *dict(arrays, positions=_t(1), wq=_t(1)).values(), *last, stream=NO_STREAM)
    assert lib.calls == 4


def test_a_view_of_the_other_kind_is_refused(lib):
    x = _t(N, C)
    with pytest.raises(ValueError):
        _call(0, q=raster.rows(x))
    with pytest.raises(ValueError):
        _call(4, x=raster.heads(_t(N, 1, C)))
    # views filled in by the caller are taken as they are
    _call(0, q=raster.gs_heads(4096, HQ * D, D))
    assert lib.calls == 1
