"""The binding of serving in 8 and 4 bits refuses arrays that a kernel would read
or write past their end: another type, too few elements, strides, host memory.
The library is replaced by one that only counts calls: nothing is launched."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from test_tokens_binding import BF16, F32, NO_STREAM, U8, CountingLibrary, _t

I8 = torch.int8
ROWS, K, N = 6, 32, 16


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
    return ((raster.gs_quantize_rows, (BF16, ROWS, K), quantize, ()),
            (raster.gs_linear_i8, (raster.linear_config(BF16, K, N), ROWS), linear, (512,)))


NAMES = [(i, name) for i, names in enumerate(("x codes scales",
                                              "x weight weight_scale bias y workspace"))
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


@pytest.mark.parametrize("i,name", NAMES)
def test_host_memory_is_refused(lib, monkeypatch, i, name):
    fn, first, arrays, last = _calls()[i]
    host = arrays[name].clone()
    monkeypatch.setattr(raster, "_on_device", lambda t: t is not host)
    with pytest.raises(ValueError):
        fn(*first, *dict(arrays, **{name: host}).values(), *last, stream=NO_STREAM)
    assert lib.calls == 0


def test_types_are_named():
    with pytest.raises(ValueError):
        raster.linear_config(torch.float64, 16, 8)
    with pytest.raises(ValueError):
        raster.gs_quantize_rows(torch.int8, 1, 16, _t(1, 16), None, None)
