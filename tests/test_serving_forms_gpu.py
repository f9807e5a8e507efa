"""The kernel instances of serving in 8 and 4 bits, against 64 bits; those that a
case is meant for are looked up in a trace of its calls, so that a changed rule
cannot move it to others unseen."""
import re

import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import Cache
from test_cached_attention_gpu import HALF, Case
from test_linear8_gpu import TYPES, _check, _normal, _run, _weights

pytestmark = pytest.mark.gpu
NAMES = {torch.float32: "float", torch.bfloat16: "Bf16", torch.float16: "F16"}


def _kernels_of(call):
    """What a call returns, and the kernels that it launches, "name type, ..."; none
    where nothing is traced."""
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as trace:
        got = call()
        torch.cuda.synchronize()
    found = set()
    for e in trace.events():
        m = re.search(r"((?:linear|cache|cached|quantize)_\w+)_kernel<([^>]*)>", e.name)
        if m:
            found.add("%s %s" % (m[1], m[2].replace("gs::", "")))
    return got, found


LINEAR = [
    (1, 2048, 8192, "linear_few", "8, true"), (1, 2048, 520, "linear_few", "16, true"),
    (8, 528, 4104, "linear_few", "8, true"), (12, 512, 520, "linear_few", "16, false"),
    (33, 144, 4096, "linear_many", "64, 32, 2, 1, 3, 4"),
    (200, 400, 4096, "linear_many", "64, 64, 2, 2, 3, 2"),
    (400, 256, 4096, "linear_many", "64, 64, 2, 2, 3, 1"),
    (1601, 144, 2056, "linear_many", "128, 128, 2, 2, 3, 1"),
    (3001, 144, 2056, "linear_many", "128, 128, 2, 2, 2, 1"),
    (5900, 144, 2040, "linear_many", "192, 256, 2, 4, 2, 1"),
    (4090, 144, 4088, "linear_many", "256, 256, 2, 4, 2, 1")]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,inputs,outputs,kernel,form", LINEAR, ids=range(len(LINEAR)))
def test_products_in_every_form(dtype, rows, inputs, outputs, kernel, form):
    x = _normal(rows, dtype, rows, inputs)
    w, ws, bias = _weights(outputs, outputs, inputs)
    y, found = _kernels_of(lambda: _run(x, w, ws, bias))
    _check(x, w, ws, bias, y)
    want = {"%s %s, %s" % (kernel, NAMES[dtype], form)}
    if "true" not in form:
        want.add("quantize_rows %s, %d" % (NAMES[dtype], 64 if inputs <= 2048 else 256))
    assert not found or found == want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim", [48, 80])
def test_caches_in_every_form(dtype, bits, dim):
    x = _normal(dim, dtype, 40, 2, dim)
    caches = [Cache(40, 2, dim, bits) for _ in range(2)]
    at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0], [40], [0], [40])]
    docs, cfg = raster.documents(*at), raster.cache_config(dtype, 2, dim)
    out = [torch.empty_like(x) for _ in range(2)]

    def call():
        views = [c.view() for c in caches]
        raster.gs_cache_write(cfg, docs, 40, 40, x, x, *views)
        raster.gs_cache_read(cfg, docs, 40, 40, *views, *out)
    _, found = _kernels_of(call)
    form = "%s, %d, %d" % (NAMES[dtype], bits, 8 if dim <= 64 else 16)
    assert not found or found == {"cache_write " + form, "cache_read " + form}
    # half a code's step; roundings of low, step, their product and sum; the type's own
    step = (x.double().amax(-1) - x.double().amin(-1)) / (2.0 ** bits - 1.0)
    most = x.double().abs().amax(-1)
    tol = 0.5 * step + 4.0 * 2.0 ** -24 * 3.0 * most + torch.finfo(dtype).eps / 2 * most
    for t in out:
        assert ((t.double() - x.double()).abs() <= tol[..., None] * (1.0 + 1e-6)).all()


SCORES = [(0, {}), (1, dict(softcap=6.0)), (1, dict(softcap=200.0)), (2, dict(slopes=True)),
          (2, dict(softcap=6.0, slopes=True)), (2, dict(softcap=200.0, slopes=True))]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dim", [48, 80])
@pytest.mark.parametrize("mode,scores", SCORES, ids=range(len(SCORES)))
def test_attention_in_every_form(dtype, bits, dim, mode, scores):
    elements = 64 if dim <= 64 else 128
    first = "%s, %d, %d" % (NAMES[dtype], bits, elements)
    # four tokens of four heads, 32 of them, and more than 128 columns
    for tokens, kernel, form in ((4, "cached_few", "1, %d" % mode), (32, "cached_few", "2, %d" % mode),
                                 (33, "cached_many", "%d" % mode)):
        c = Case(dtype, bits, 4, 1, dim, [tokens, 1], [tokens + 300, 77], **scores)
        got, found = _kernels_of(c.run)
        c.check(*got)
        assert not found or "%s %s, %s" % (kernel, first, form) in found, found
    if mode == 2:
        return
    # behind a shared prompt, each with each
    for own in (1, 9, 70):
        for many in (1, 8):
            c = Case(dtype, bits, 4, 1, dim, [own] * many, [own + 40 * i for i in range(many)],
                     shared=[(0, many, 333)], **scores)
            got, found = _kernels_of(c.run)
            c.check(*got)
            assert not found or "cached_both %s, %d" % (first, mode) in found, found


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [48, 80])
@pytest.mark.parametrize("keys,threads", [(700, 64), (4000, 64), (6000, 256)])
def test_joins_in_every_form(dtype, dim, keys, threads):
    c = Case(dtype, 8, 2, 1, dim, [1, 3], [keys, 500])
    got, found = _kernels_of(c.run)
    c.check(*got)
    lanes = 16 if dim <= 64 else 32
    assert not found or "cached_join %s, %d, %d" % (NAMES[dtype], lanes, threads) in found, found
    # one piece: nothing to join
    c = Case(dtype, 8, 2, 1, dim, [1, 3], [200, 90])
    got, found = _kernels_of(c.run)
    c.check(*got)
    assert not any("join" in name for name in found)
