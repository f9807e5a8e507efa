"""Rows brought to 8 bits, and products with 8-bit weights, against 64 bits."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import linear, linear_error, row_codes
from token_util import close

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


def _normal(seed, dtype, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _space(n):
    return torch.empty((max(n, 256),), dtype=torch.uint8, device="cuda")


def _weights(seed, outputs, inputs, bias=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(-127, 128, (outputs, inputs), generator=gen, device="cuda",
                      dtype=torch.int8)
    return (w, torch.rand(outputs, generator=gen, device="cuda") * 0.01 + 0.001,
            torch.randn(outputs, generator=gen, device="cuda") if bias else None)


def _run(x, w, ws, bias, y=None, stream=None):
    cfg = raster.linear_config(x.dtype, w.shape[1], w.shape[0])
    if y is None:
        y = torch.full((x.shape[0], w.shape[0]), 7.0, dtype=x.dtype, device="cuda")
    n = raster.gs_linear_i8_workspace_size(cfg, x.shape[0])
    raster.gs_linear_i8(cfg, x.shape[0], x, w, ws, bias, y, _space(n), n, stream=stream)
    return y


def _check(x, w, ws, bias, y):
    want, size = linear(x, w, ws, bias)
    # past the type's largest number (1.5e39 in fp32) the nearest is infinity
    over = want.abs() > torch.finfo(x.dtype).max
    assert torch.equal(y[over].double(), want[over].sign() * INF)
    bad = torch.isnan(want) | over
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    zero = torch.zeros_like(want)
    close(torch.where(bad, torch.zeros_like(y), y), torch.where(bad, zero, want),
          torch.where(bad, zero, linear_error(want, size, x.dtype)), "y")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,channels", [(1, 16), (3, 48), (5, 512), (7, 2048), (2, 2064),
                                           (9, 8192), (3, 8208), (2, 20016), (700, 80)])
def test_rows_to_8_bits(dtype, rows, channels):
    wide = _normal(rows + channels, dtype, rows, channels + 24)
    x = wide[:, 8:8 + channels]
    x *= torch.logspace(-4, 4, rows, device="cuda")[:, None].to(dtype)
    codes = torch.full((rows, channels), 99, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    raster.gs_quantize_rows(dtype, rows, channels, x, codes, scales)
    want, scale = row_codes(x)
    assert torch.equal(codes.double(), want)
    assert torch.equal(scales, scale.float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("channels", [64, 4096])
def test_rows_without_codes(dtype, channels):
    x = _normal(3, dtype, 9, channels)
    x[0] = 0.0
    x[1, 5], x[2, 7], x[3, channels - 1] = NAN, INF, -INF
    x[4] = 0.0
    x[4, 9] = 2.0 ** -120 if dtype != torch.float16 else 2.0 ** -24
    x[5] = 2.0 ** -115 if dtype != torch.float16 else 6e4
    x[6] = torch.finfo(dtype).max
    x[6, ::2] = -torch.finfo(dtype).max
    x[7, 0], x[8, :] = NAN, NAN
    codes = torch.empty((9, channels), dtype=torch.int8, device="cuda")
    scales = torch.empty(9, device="cuda")
    raster.gs_quantize_rows(dtype, 9, channels, x, codes, scales)
    want, scale = row_codes(x)
    assert torch.equal(codes.double(), want)
    assert torch.equal(torch.nan_to_num(scales, nan=-1.0), torch.nan_to_num(scale.float(), nan=-1.0))
    w, ws, bias = _weights(1, 24, channels)
    _check(x, w, ws, bias, _run(x, w, ws, bias))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,inputs,outputs", [
    (1, 16, 8), (1, 64, 16), (1, 2048, 520), (2, 80, 24), (15, 144, 40), (16, 1040, 72),
    (17, 512, 16), (31, 336, 136), (33, 2064, 264), (64, 96, 8), (65, 128, 128),
    (65, 16, 8), (129, 144, 136), (200, 400, 264), (257, 1024, 8), (1000, 272, 1032)])
def test_products(dtype, rows, inputs, outputs):
    x = _normal(rows, dtype, rows, inputs)
    w, ws, bias = _weights(outputs, outputs, inputs, rows % 2 == 1)
    _check(x, w, ws, bias, _run(x, w, ws, bias))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,inputs,outputs", [(4096, 144, 4096), (4093, 400, 4104),
                                                 (2049, 128, 8200), (16000, 2064, 1288)])
def test_large_products(dtype, rows, inputs, outputs):
    x = _normal(rows, dtype, rows, inputs)
    w, ws, bias = _weights(outputs, outputs, inputs)
    _check(x, w, ws, bias, _run(x, w, ws, bias))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("inputs", [16, 144, 272, 656, 1552])
@pytest.mark.parametrize("rows,outputs", [(1601, 2056), (3001, 2056), (5900, 2040), (4090, 4088),
                                          (10, 4104), (40, 1032), (64, 8), (190, 4088),
                                          (600, 2056)])
def test_products_of_few_steps_in_each_tile(dtype, rows, outputs, inputs):
    """128 by 128 outputs with two steps ahead and with one, 192 by 256, 256 by 256, 64 by
    32 with the steps in four parts, 64 by 64 in two and in one."""
    x = _normal(rows + inputs, dtype, rows, inputs)
    w, ws, bias = _weights(outputs, outputs, inputs, inputs != 272)
    _check(x, w, ws, bias, _run(x, w, ws, bias))


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_sums_at_their_ends(rows):
    """All codes at the ends of their range and inputs at their most: sums near
    2^31 are exact."""
    inputs, outputs = 131056, 16
    x = torch.ones((rows, inputs), dtype=torch.bfloat16, device="cuda")
    x[::2] = -1.0
    w = torch.full((outputs, inputs), 127, dtype=torch.int8, device="cuda")
    w[::3] = -127
    ws = torch.full((outputs,), 2.0 ** -20, device="cuda")
    _check(x, w, ws, None, _run(x, w, ws, None))


@pytest.mark.parametrize("rows", [1, 20, 50, 140, 3000])
def test_strides_and_rows_between(rows):
    wide = _normal(rows, torch.bfloat16, rows, 400)
    out = torch.full((rows + 2, 328), 5.0, dtype=torch.bfloat16, device="cuda")
    w, ws, bias = _weights(3, 264, 272)
    x, y = wide[:, 64:336], out[:rows, 32:296]
    _run(x, w, ws, bias, y)
    _check(x, w, ws, bias, y)
    assert (out[rows:] == 5.0).all() and (out[:, :32] == 5.0).all() and (out[:, 296:] == 5.0).all()
    # the same rows many times over
    same = wide[:1, 64:336].expand(rows, 272)
    if rows > 1:
        _check(same, w, ws, bias, _run(same, w, ws, bias))


@pytest.mark.parametrize("rows", [1, 33, 700])
def test_same_bits_on_a_stream_and_in_a_graph(rows):
    x = _normal(rows, torch.float16, rows, 1024)
    w, ws, bias = _weights(4, 512, 1024)
    want = _run(x, w, ws, bias).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = _run(x, w, ws, bias, stream=side)
    side.synchronize()
    assert torch.equal(want, other)
    cfg = raster.linear_config(x.dtype, 1024, 512)
    n = raster.gs_linear_i8_workspace_size(cfg, rows)
    space, y = _space(n), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        raster.gs_linear_i8(cfg, rows, x, w, ws, bias, y, space, n)
    for i in range(4):
        x.copy_(_normal(50 + i, torch.float16, rows, 1024))
        y.zero_()
        space.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, _run(x, w, ws, bias))


def test_no_rows():
    w, ws, bias = _weights(1, 8, 16)
    _run(torch.empty((0, 16), device="cuda"), w, ws, bias)
