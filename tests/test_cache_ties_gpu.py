"""Codes of a cache next to ties, where 64-bit quotients cannot tell, against
exact fractions."""
from fractions import Fraction

import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import Cache, pack

pytestmark = pytest.mark.gpu


def _exact(head, bits):
    """Codes of a head by the formula: to the nearest, to even at a tie."""
    x = [Fraction(v) for v in head]
    low, levels = min(x), 2 ** bits - 1
    span = max(x) - low
    return [round(levels * (v - low) / span) for v in x]       # Fraction's round: to even


def _write(x, bits):
    """The caches of tokens x [rows, heads, dim] as keys, and reversed as values."""
    rows, heads, dim = x.shape
    caches = [Cache(rows, heads, dim, bits) for _ in range(2)]
    at = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0], [rows], [0], [rows])]
    raster.gs_cache_write(raster.cache_config(x.dtype, heads, dim), raster.documents(*at), rows,
                          rows, x, x.flip(-1), *[c.view() for c in caches])
    return caches


LOWS = {torch.float16: [0.0, 2.0 ** -24, 2.0 ** -23, 2.0 ** -14],
        torch.bfloat16: [0.0] + [2.0 ** -n for n in (6, 24, 30, 33, 40, 60, 100, 126)],
        torch.float32: [0.0] + [2.0 ** -n for n in (6, 24, 30, 33, 40, 60, 100, 126, 149)]}


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", list(LOWS))
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("sign", [1, -1])
def test_next_to_ties(dtype, bits, dim, sign):
    """From 0 to twice the levels every odd number is a tie; a smallest element a
    little off 0 puts it to one side, by up to 2^-149."""
    levels = 2 ** bits - 1
    size = 1.0
    if dtype == torch.float16:   # up to 2^15, so that its smallest number is far below
        size = 64.0 if bits == 8 else 1024.0
    rng = torch.Generator().manual_seed(dim + bits)
    heads = []
    for low in LOWS[dtype]:
        for _ in range(4):
            # bf16 holds odd numbers up to 255
            odd = 2 * torch.randint(0, min(levels, 128), (dim,), generator=rng) + 1.0
            odd[torch.randint(0, dim, (dim // 8,), generator=rng)] *= 0.75
            place = torch.randperm(dim, generator=rng)
            odd[place[:3]] = torch.tensor([2.0 * levels, 0.0, 2.0 * levels - 1.0])
            odd *= size
            odd[place[1]] = sign * low
            heads.append(odd)
    x = torch.stack(heads).to(dtype)
    want = torch.tensor([_exact(h, bits) for h in x.double().tolist()])
    for cache, w in zip(_write(x.cuda()[:, None], bits), (want, want.flip(-1))):
        assert torch.equal(cache.codes[:, 0].cpu(), pack(w, bits).view(len(x), -1))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", list(LOWS))
def test_random_heads_of_wide_range(dtype, bits):
    """Elements of all exponents, and of few different ones, which meet ties often."""
    rng = torch.Generator().manual_seed(bits)
    wide = torch.randn((24, 48), generator=rng) * 2.0 ** torch.randint(-20, 14, (24, 48), generator=rng)
    few = torch.randint(-9, 10, (40, 48), generator=rng) * 2.0 ** torch.randint(-3, 4, (40, 1), generator=rng)
    x = torch.cat((wide, few)).to(dtype)
    want = torch.tensor([_exact(h, bits) for h in x.double().tolist()])
    cache = _write(x.cuda()[:, None], bits)[0]
    assert torch.equal(cache.codes[:, 0].cpu(), pack(want, bits).view(len(x), -1))


@pytest.mark.parametrize("bits", [8, 4])
def test_the_widest_heads(bits):
    """Spans next to 2^127: below it codes, also where fp32 rounds the span to it."""
    top = 2.0 ** 126
    below = top - 2.0 ** 102                                   # the next fp32 number
    x = torch.randn((3, 1, 16), generator=torch.Generator().manual_seed(bits)) * 2.0 ** 120
    x[0, 0, 3], x[0, 0, 7] = top, -below
    x[1, 0, 3], x[1, 0, 7] = top, -top
    x[2, 0, 3], x[2, 0, 7] = below, -below
    cache = _write(x.cuda(), bits)[0]
    want = torch.tensor([_exact(x[i, 0].double().tolist(), bits) if i != 1 else [0] * 16
                         for i in range(3)])
    assert torch.equal(cache.codes[:, 0].cpu(), pack(want, bits).view(3, -1))
    assert torch.isnan(cache.low[0, 1]) and torch.isnan(cache.step[0, 1])
    for i in (0, 2):
        span = x[i].double().max() - x[i].double().min()
        assert float(cache.low[0, i]) == -below
        assert float(cache.step[0, i]) == float((span / (2 ** bits - 1)).float())
