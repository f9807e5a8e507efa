"""Attention over caches whose steps differ much in size or in sign, against 64 bits."""
import pytest
import torch

import test_cached_attention_gpu as base
from serving_util import U, Cache, cached_head
from test_cached_attention_gpu import HALF, Case
from token_util import close

pytestmark = pytest.mark.gpu
# tokens of a document, of four query heads over one key head: 16, 32 and 128 columns
FORMS = [1, 9, 70]


class Turned(Cache):
    """A cache whose heads may count downwards.  parts() gives them upwards: the
    same numbers, and what serving_util's bounds ask for."""

    def parts(self, rows, head):
        u, low, step = super().parts(rows, head)
        most = 2.0 ** self.bits - 1.0
        down = step < 0
        return (torch.where(down[:, None], most - u, u), torch.where(down, low + most * step, low),
                step.abs())

    def turn(self, which):
        """Rows `which` downwards, near the numbers that they hold."""
        self.low[:, which] += (2.0 ** self.bits - 1.0) * self.step[:, which]
        self.step[:, which] *= -1.0
        self.codes[which] = self.codes[which] ^ 255


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("all_down", [False, True])
def test_heads_that_count_downwards(monkeypatch, dtype, bits, dim, own, shared, all_down):
    """low + step code with a negative step, in some rows and in all."""
    c = Case(dtype, bits, 4, 1, dim, [own, 2], [own + 140, 37],
             shared=[(0, 2, 300)] if shared else ())
    rows = torch.arange(c.rows_k, device="cuda")
    for t in (c.k, c.v):
        t.__class__ = Turned
        t.turn(rows if all_down else rows[rows % 3 != 0])
    # a head that counts down has its codes on the other side of the middle: up to one
    # step more that is rounded to half a step of fp16, for weights whose sum is 1
    more = (2.0 ** -11 + 2.0 ** -12) * float(c.v.step.abs().max())
    monkeypatch.setattr(base, "close", lambda got, want, tol, what: close(
        got, want, tol + (more if what == "o" else 0.0), what))
    c.check(*c.run())


def _positive(c):
    """Queries of positive elements, so that a key of one number has the score it says."""
    c.q = (0.5 + 0.5 * c.q.abs()).to(c.dtype)
    return c


def _plain_key(c, row, number):
    c.k.codes[row], c.k.low[:, row], c.k.step[:, row] = 0, number, 0.0


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own", [2, 4, 9, 40, 70])
@pytest.mark.parametrize("shared", [False, True])
def test_large_steps_that_later_tokens_see(dtype, bits, dim, own, shared):
    """A token's result is the same bits whatever finite numbers stand in keys that
    only later tokens of its document see."""
    c = Case(dtype, bits, 4, 1, dim, [own, 3], [own + 75, 50],
             shared=[(0, 2, 300)] if shared else ())
    want = c.run()
    half, end = own // 2, c.k_starts[0] + c.k_lens[0]
    rows = torch.arange(end - own + half, end, device="cuda")
    for factor in (2.0 ** 20, 1e20, -1e28):
        for t in (c.k, c.v):
            keep = t.low[:, rows].clone(), t.step[:, rows].clone()
            t.low[:, rows] *= factor
            t.step[:, rows] *= factor
            got = c.run()
            t.low[:, rows], t.step[:, rows] = keep
            seen = list(range(c.q_starts[0], c.q_starts[0] + half)) + \
                list(range(c.q_starts[1], c.q_starts[1] + 3))
            assert torch.equal(got[0][seen], want[0][seen])
            assert torch.equal(got[1][:, seen], want[1][:, seen])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own", FORMS)
def test_large_steps_without_weight(dtype, bits, dim, own):
    """A value whose weight is zero does not matter, however large its step."""
    c = _positive(Case(dtype, bits, 4, 1, dim, [own], [own + 140]))
    row = c.k_starts[0] + 40
    _plain_key(c, row, -100.0)          # a score of -500 or less
    want = c.run()
    for step in (2.0 ** 40, 2.0 ** 90, -2.0 ** 90):
        c.v.step[:, row] = step
        got = c.run()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def _by_weight(q, key, value, scale, softcap, slope, seen, away, bits, dtype):
    """serving_util's bound, but that of fp16's smallest numbers: they are relative to
    the token's largest product of weight and step, not to the largest step."""
    o, tol, lse, e_lse = cached_head(q, key, value, scale, softcap, slope, seen, away, bits, dtype)
    k = key[1][:, None] + key[2][:, None] * key[0]
    s = (q @ k.T * scale).masked_fill(~seen, float("-inf"))
    p, step = torch.exp(s - lse[:, None]), value[2]
    each = 2.0 ** -33 * seen.double().sum(1, keepdim=True) * 2.0 ** bits
    less = each * (step.max() - (p * step).amax(1, keepdim=True))
    return o, tol - (1.0 + U[dtype]) * less, lse, e_lse


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own", FORMS)
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("how", ["faint", "past"])
def test_large_steps_with_little_weight(monkeypatch, dtype, bits, dim, own, shared, how):
    """A value of step 2^30 (fp16: its result stays below the type's end), whose key
    has a score of about -40, or one of 0 before later keys of about 100."""
    c = _positive(Case(dtype, bits, 4, 1, dim, [own], [own + 140],
                       shared=[(0, 1, 300)] if shared else ()))
    at = c.k_starts[0]
    if how == "faint":
        _plain_key(c, at + 40, -5.0)
        c.v.step[:, at + 40] = 2.0 ** 30
    else:
        c.v.step[:, at + 3] = 2.0 ** 30
        for i in range(5):
            _plain_key(c, at + 100 + i, 15.0)
    monkeypatch.setattr(base, "cached_head", _by_weight)
    c.check(*c.run())


@pytest.mark.parametrize("bits", [8, 4])
def test_many_large_values(bits):
    """2^17 values of 2^99, whose keys' scores rise after the first of each piece: the
    sum of the values is 2^116, that of the weights is held relative to a score."""
    n = 1 << 17
    c = Case(torch.bfloat16, bits, 1, 1, 16, [1], [n])
    rows = torch.arange(c.k_starts[0], c.k_starts[0] + n, device="cuda")
    c.q.fill_(1.0)
    _plain_key(c, rows, torch.where((rows - c.k_starts[0]) % 512 < 128, 0.0, 1.02))
    c.v.low[:, rows], c.v.step[:, rows] = 2.0 ** 99, 0.0
    out, _ = c.run()
    token = out[c.q_starts[0]].double()
    # fp32 sums of n numbers in chains of a lane each, and the type's rounding
    assert ((token / 2.0 ** 99 - 1.0).abs() <= 2.0 ** -8 + (n / 128 + 16) * 2.0 ** -24).all()
