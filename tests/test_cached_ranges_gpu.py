"""Attention over caches whose steps differ much in size or in sign, against 64 bits."""
import pytest
import torch

import test_cached_attention_gpu as base
from serving_util import Cache
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
