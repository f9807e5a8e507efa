"""Products of up to eight rows, which are brought to 8 bits inside the product:
every partition of a workgroup's wavefronts over the rows, up to the ends of what it
takes, against 64 bits."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import linear, linear_error
from test_linear8_gpu import INF, NAN, TYPES, _normal, _run, _weights
from token_util import close

pytestmark = pytest.mark.gpu

# up to 4,096 outputs a workgroup has 16 wavefronts, else 8; a wavefront has 512
# elements of a row at a time, four times at most
LIMIT = 96 << 20  # elements that all workgroups together bring to codes


def _sizes(rows, outputs):
    """Inputs that end in the first, second and fourth piece of a lane's elements
    where the call takes as many, and the most that it takes."""
    shares = rows if rows <= 2 else 4 if rows <= 4 else 8
    piece = (16 if outputs <= 4096 else 8) // shares * 512
    most = min(4 * piece, LIMIT // (shares * outputs)) // 16 * 16
    return [n for n in (piece // 2 + 16, piece + 208, 3 * piece + 400) if n < most] + [most]


def _inside(dtype, rows, inputs, outputs):
    """Whether the rows are brought to codes without a launch, and a place, of their own."""
    cfg = raster.linear_config(dtype, inputs, outputs)
    return raster.gs_linear_i8_workspace_size(cfg, rows) == 0


def _check(x, w, ws, bias, y):
    want, size = linear(x, w, ws, bias)
    tol = linear_error(want, size, x.dtype)
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    # A type of p bits ends with (2 - 2^(1 - p)) 2^e; numbers up to half a step, 2^(e - p),
    # past that are rounded to it, others to infinity: in fp16 65,520 is the first of these.
    info = torch.finfo(x.dtype)
    end = info.max + info.max / (2.0 - info.eps) * info.eps / 2.0
    past, near = want.abs() - tol > end, (want.abs() - end).abs() <= tol
    assert torch.equal(y[past].double(), want[past].sign() * INF)
    edge = y[near].double()
    assert ((edge.abs() >= info.max) & (edge.sign() == want[near].sign())).all()
    rest = ~(past | near | torch.isnan(want))
    close(y[rest], want[rest], tol[rest], "y")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("outputs", [520, 4064, 4104])
def test_rows_brought_to_8_bits_inside(dtype, rows, outputs):
    sizes = _sizes(rows, outputs)
    for inputs in sizes + [sizes[-1] + 16]:
        assert _inside(dtype, rows, inputs, outputs) == (inputs <= sizes[-1])
        x = _normal(rows + inputs, dtype, rows, inputs + 8)[:, :inputs]
        x *= torch.logspace(-3, 3, rows, device="cuda")[:, None].to(dtype)
        # the largest magnitude in the last piece, in every one, and anywhere
        x[0, -1] = 4.5 * x[0].abs().max()
        w, ws, bias = _weights(inputs, outputs, inputs, rows % 2 == 1)
        _check(x, w, ws, bias, _run(x, w, ws, bias))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("outputs", [24, 4104])
@pytest.mark.parametrize("first", range(8))
@pytest.mark.parametrize("rows", [1, 3, 8])
def test_rows_without_codes_inside(dtype, outputs, first, rows):
    """Zeros, tiny and largest numbers, infinities and NaN, in turn over the rows."""
    inputs = 1552
    top = torch.finfo(dtype).max
    x = _normal(first, dtype, 8, inputs)
    x[0] = 0.0
    x[1, 5], x[2, 700], x[3, inputs - 1] = NAN, INF, -INF
    x[4] = 0.0
    x[4, 9] = 2.0 ** -120 if dtype != torch.float16 else 2.0 ** -24
    x[5] = 2.0 ** -115 if dtype != torch.float16 else 6e4
    x[6], x[6, ::2] = top, -top
    x[7, 0], x[7, 1], x[7, 1000] = INF, -NAN, -INF
    x = x.roll(-first, 0)[:rows].contiguous()
    w, ws, bias = _weights(first, outputs, inputs)
    assert _inside(dtype, rows, inputs, outputs)
    _check(x, w, ws, bias, _run(x, w, ws, bias))
