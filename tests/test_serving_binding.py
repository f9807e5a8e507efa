"""The binding of serving in 8 and 4 bits refuses arrays that a kernel would read
or write past their end: another type, too few elements, strides, host memory.
The library is replaced by one that only counts calls: nothing is launched."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from test_tokens_binding import BF16, F32, NO_STREAM, U8, CountingLibrary, _t

I8, I32 = torch.int8, torch.int32
ROWS, K, N = 6, 32, 16
H, D, HELD, DOCS = 2, 32, 20, 3


def _cache(rows=HELD, heads=H, dim=D, bits=4):
    planes = [_t(heads, rows, dtype=F32) for _ in range(2)]
    return raster.codes(_t(rows, heads, dim * bits // 8, dtype=U8), *planes, bits)


@pytest.fixture
def lib(monkeypatch):
    lib = CountingLibrary()
    monkeypatch.setattr(raster, "_lib", lib)
    # host tensors stand in for device memory here
    monkeypatch.setattr(raster, "_on_device", lambda t: True)
    return lib


def _calls():
    x, w = _t(ROWS, K), _t(N, K, dtype=I8)
    quantize = dict(x=x, codes=_t(ROWS, K, dtype=I8), scales=_t(ROWS, dtype=F32))
    linear = dict(x=x, weight=w, weight_scale=_t(N, dtype=F32), bias=_t(N, dtype=F32),
                  y=_t(ROWS, N), workspace=_t(512, dtype=U8))
    docs = raster.documents(*[_t(DOCS, dtype=I32) for _ in range(4)])
    k, q, lse = _t(ROWS, H, D), _t(ROWS, 2 * H, D), _t(2 * H, ROWS, dtype=F32)
    write = dict(k=k, v=k, k_cache=_cache(), v_cache=_cache())
    read = dict(k_cache=_cache(), v_cache=_cache(), k=k, v=k)
    attend = dict(q=q, k_cache=_cache(), v_cache=_cache(), out=q, lse=lse,
                  workspace=_t(512, dtype=U8))
    cfg = raster.cache_config(BF16, H, D)
    at_cfg = raster.attention_config(BF16, 2 * H, H, D, 0.1)
    return ((raster.gs_quantize_rows, (BF16, ROWS, K), quantize, ()),
            (raster.gs_linear_i8, (raster.linear_config(BF16, K, N), ROWS), linear, (512,)),
            (raster.gs_cache_write, (cfg, docs, ROWS, HELD), write, ()),
            (raster.gs_cache_read, (cfg, docs, ROWS, HELD), read, ()),
            (raster.gs_cached_attention_fwd, (at_cfg, docs, docs, ROWS, HELD), attend, (512,)))


NAMES = [(i, name) for i, names in enumerate(("x codes scales",
                                              "x weight weight_scale bias y workspace",
                                              "k v k_cache v_cache", "k_cache v_cache k v",
                                              "q k_cache v_cache out lse workspace"))
         for name in names.split()]
ARRAYS = [(i, name) for i, name in NAMES if not name.endswith("cache")]


def _call(i, **other):
    fn, first, arrays, last = _calls()[i]
    fn(*first, *dict(arrays, **other).values(), *last, stream=NO_STREAM)


@pytest.mark.parametrize("i,name", ARRAYS)
def test_arrays_that_do_not_fit_are_refused(lib, i, name):
    _call(i)
    assert lib.calls == 1
    assert list(_calls()[i][2]) == [n for j, n in NAMES if j == i]
    t = _calls()[i][2][name]
    bad = [t[:-1].clone()]                                       # too few
    if t.dtype != U8:
        bad += [t.to(torch.float16), t.to(torch.float64)]        # another type
        bad.append(t[..., :-8].contiguous())                     # shorter rows
    if t.dtype != BF16:
        bad.append(torch.zeros_like(t[:1]).expand(t.shape))      # no memory behind it
    for b in bad:
        with pytest.raises(ValueError):
            _call(i, **{name: b})
    assert lib.calls == 1


@pytest.mark.parametrize("i,name", ARRAYS)
def test_host_memory_is_refused(lib, monkeypatch, i, name):
    fn, first, arrays, last = _calls()[i]
    host = arrays[name].clone()
    monkeypatch.setattr(raster, "_on_device", lambda t: t is not host)
    with pytest.raises(ValueError):
        fn(*first, *dict(arrays, **{name: host}).values(), *last, stream=NO_STREAM)
    assert lib.calls == 0


@pytest.mark.parametrize("i", [2, 3, 4])
@pytest.mark.parametrize("name", ["k_cache", "v_cache"])
def test_caches_that_do_not_fit_are_refused(lib, i, name):
    for bad in (_cache(rows=HELD - 1), _cache(heads=H - 1), _cache(dim=D - 16), None,
                _t(HELD, H, D // 2, dtype=U8)):
        with pytest.raises(ValueError):
            _call(i, **{name: bad})
    assert lib.calls == 0
    _call(i, **{name: _cache(rows=HELD + 1, heads=H + 1, dim=D + 16)})
    # a cache filled in by the caller is taken as it is
    _call(i, **{name: raster.gs_codes(4096, 4096, 4096, 64, 32, 20, 4)})
    assert lib.calls == 2


def test_arrays_of_a_cache_are_checked(lib, monkeypatch):
    def make(codes=_t(5, 2, 32, dtype=U8), low=_t(2, 5, dtype=F32), step=_t(2, 5, dtype=F32),
             bits=8):
        return raster.codes(codes, low, step, bits)
    c = make()
    assert (c.row, c.head, c.ld, c.bits, c.extent) == (64, 32, 5, 8, (5, 2, 32))
    c = make(_t(2, 5, 32, dtype=U8).transpose(0, 1), _t(2, 9, dtype=F32)[:, :5],
             _t(2, 9, dtype=F32)[:, 4:], bits=4)
    assert (c.row, c.head, c.ld, c.extent) == (32, 160, 9, (5, 2, 64))
    for bad in (dict(bits=2), dict(codes=_t(5, 2, 32)), dict(codes=_t(5, 64, dtype=U8)),
                dict(codes=_t(5, 32, 2, dtype=U8).transpose(1, 2)), dict(low=_t(2, 4, dtype=F32)),
                dict(low=_t(2, 5)), dict(step=_t(5, 2, dtype=F32).T), dict(step=_t(2, 6, dtype=F32)),
                dict(low=_t(2, 9, dtype=F32)[:, :5])):
        with pytest.raises(ValueError):
            make(**bad)
    monkeypatch.setattr(raster, "_on_device", lambda t: False)
    with pytest.raises(ValueError):
        make()


class Elsewhere:
    """A tensor as if it were on a device."""

    def __init__(self, t, device):
        self.t, self.device_index = t, device

    def get_device(self):
        return self.device_index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("i,name", ARRAYS)
def test_tensors_of_another_device_are_refused(lib, monkeypatch, i, name):
    import types
    t = _calls()[i][2][name]
    fn, first, arrays, last = _calls()[i]
    call = lambda there, here: fn(*first, *dict(arrays, **{name: Elsewhere(t, there)}).values(),
                                  *last, stream=types.SimpleNamespace(cuda_stream=0,
                                                                      device_index=here))
    monkeypatch.setattr(raster, "_devices", 2)
    with pytest.raises(ValueError):
        call(1, 0)
    assert lib.calls == 0
    call(1, 1)
    call(-1, 0)                                                  # page-locked
    monkeypatch.setattr(raster, "_devices", 1)
    call(1, 0)
    assert lib.calls == 3


def test_a_cache_of_another_device_is_refused(lib, monkeypatch):
    import types
    monkeypatch.setattr(raster, "_devices", 2)
    fn, first, arrays, last = _calls()[2]
    c = _cache()
    c.tensors = tuple(Elsewhere(t, 1) for t in c.tensors)
    stream = types.SimpleNamespace(cuda_stream=0, device_index=0)
    with pytest.raises(ValueError):
        fn(*first, *dict(arrays, k_cache=c).values(), *last, stream=stream)
    assert lib.calls == 0


def test_slopes_of_another_device_are_refused(lib, monkeypatch):
    import types
    monkeypatch.setattr(raster, "_devices", 2)
    fn, first, arrays, last = _calls()[4]
    first[0].tensor = Elsewhere(torch.zeros(first[0].heads_q), 1)
    stream = types.SimpleNamespace(cuda_stream=0, device_index=0)
    with pytest.raises(ValueError):
        fn(*first, *arrays.values(), *last, stream=stream)
    assert lib.calls == 0


def test_types_are_named():
    with pytest.raises(ValueError):
        raster.linear_config(torch.float64, 16, 8)
    with pytest.raises(ValueError):
        raster.gs_quantize_rows(torch.int8, 1, 16, _t(1, 16), None, None)
