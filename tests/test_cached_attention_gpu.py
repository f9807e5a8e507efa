"""Attention over caches of 8 and 4 bits against 64 bits."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import Cache, cached_head
from token_util import close

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


class Case:
    """Documents over one cache: q_lens and k_lens, shared: (first document, number,
    keys) of each shared prefix."""

    def __init__(self, dtype, bits, heads_q, heads_k, dim, q_lens, k_lens, shared=(), seed=0,
                 gap=3, causal=True, softcap=0.0, slopes=False, prefix=None, spread=1.0,
                 head_major=False, tight=False):
        self.dtype, self.bits, self.hq, self.hk, self.dim = dtype, bits, heads_q, heads_k, dim
        self.q_lens, self.k_lens, self.shared = list(q_lens), list(k_lens), list(shared)
        self.causal, self.softcap, self.prefix = causal, softcap, prefix
        at = gap
        self.p_starts = []
        for _, _, n in self.shared:
            self.p_starts.append(at)
            at += n + gap
        self.k_starts = []
        for n in self.k_lens:
            self.k_starts.append(at)
            at += n + gap
        # tight: the cache ends with the last document
        self.rows_k = max(at - gap, 1) if tight else at
        self.q_starts, at = [], 1 if self.q_lens else 0
        for i, n in enumerate(self.q_lens):
            self.q_starts.append(at)
            at += n
        self.rows_q = at + 2
        scale = torch.logspace(-0.5, 0.5, self.rows_k, device="cuda")[:, None, None] ** spread
        mean = 0.4 * _normal(seed + 5, heads_k, dim)
        self.k = Cache(self.rows_k, heads_k, dim, bits, head_major=head_major, spare=16)
        self.v = Cache(self.rows_k, heads_k, dim, bits, head_major=head_major)
        self.k.fill(_normal(seed + 1, self.rows_k, heads_k, dim) + mean)
        self.v.fill((_normal(seed + 2, self.rows_k, heads_k, dim) + mean) * scale)
        self.q = _normal(seed + 3, self.rows_q, heads_q + 1, dim).to(dtype)[:, 1:]
        self.scale = dim ** -0.5
        self.slopes = 2.0 ** -(1.0 + torch.arange(heads_q, device="cuda")) if slopes else None
        self.cfg = raster.attention_config(dtype, heads_q, heads_k, dim, self.scale, causal,
                                           softcap, self.slopes)

    def documents(self, hints=True):
        h = dict(max_q_len=max(self.q_lens, default=0), max_k_len=max(self.k_lens, default=0))
        if hints is not True:
            h = dict(max_q_len=hints[0], max_k_len=hints[1])
        docs = raster.documents(*map(_ints, (self.q_starts, self.q_lens, self.k_starts,
                                             self.k_lens)),
                                prefix=None if self.prefix is None else _ints(self.prefix), **h)
        if not self.shared:
            return docs, None
        starts, lens, keys = [], [], []
        for first, n, k in self.shared:
            starts.append(self.q_starts[first])
            lens.append(sum(self.q_lens[first:first + n]))
            keys.append(k)
        h = dict(max_q_len=max(lens), max_k_len=max(keys))
        if hints is not True:
            h = dict(max_q_len=hints[0], max_k_len=hints[1])
        return docs, raster.documents(*map(_ints, (starts, lens, self.p_starts, keys)), **h)

    def run(self, hints=True, lse=True, stream=None):
        docs, shared = self.documents(hints)
        out = torch.full((self.rows_q, self.hq + 1, self.dim), 9.0, dtype=self.dtype,
                         device="cuda")[:, 1:]
        sums = torch.full((self.hq, self.rows_q), 9.0, device="cuda") if lse else None
        n = raster.gs_cached_attention_fwd_workspace_size(self.cfg, self.bits, docs, shared,
                                                          self.rows_q, self.rows_k)
        space = torch.full((max(n, 256),), 255, dtype=torch.uint8, device="cuda")
        raster.gs_cached_attention_fwd(self.cfg, docs, shared, self.rows_q, self.rows_k, self.q,
                                       self.k.view(), self.v.view(), out, sums, space, n,
                                       stream=stream)
        return out, sums

    def check(self, out, lse):
        want = torch.full(out.shape, 9.0, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        sums = torch.full((self.hq, self.rows_q), 9.0, dtype=torch.float64, device="cuda")
        e_sums = torch.zeros_like(sums)
        group = self.hq // self.hk
        for d, (q0, nq, k0, nk) in enumerate(zip(self.q_starts, self.q_lens, self.k_starts,
                                                 self.k_lens)):
            if nq == 0:
                continue
            front = [list(range(p, p + n)) for p, (first, m, n) in zip(self.p_starts, self.shared)
                     if first <= d < first + m]
            front = front[0] if front else []
            rows = torch.tensor(front + list(range(k0, k0 + nk)), dtype=torch.long, device="cuda")
            i = torch.arange(nq, device="cuda")[:, None] + nk - nq
            j = torch.arange(nk, device="cuda")[None, :]
            seen = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
            if self.causal:
                seen = (j <= i) | (j < (self.prefix[d] if self.prefix else 0))
            seen = torch.cat((torch.ones((nq, len(front)), dtype=torch.bool, device="cuda"), seen),
                             1)
            away = torch.cat((torch.zeros((nq, len(front)), device="cuda"), (i - j).abs()),
                             1).double()
            for h in range(self.hq):
                o, eo, s, es = cached_head(
                    self.q[q0:q0 + nq, h].double(), self.k.parts(rows, h // group),
                    self.v.parts(rows, h // group), self.scale, self.softcap,
                    0.0 if self.slopes is None else float(self.slopes[h]), seen, away, self.bits,
                    self.dtype)
                want[q0:q0 + nq, h], tol[q0:q0 + nq, h] = o, eo
                sums[h, q0:q0 + nq], e_sums[h, q0:q0 + nq] = s, es
        close(out, want, tol, "o")
        if lse is not None:
            none = torch.isinf(sums)
            assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all()
            close(torch.where(none, torch.zeros_like(lse), lse),
                  torch.where(none, torch.zeros_like(sums), sums),
                  torch.where(none, torch.zeros_like(sums), e_sums), "lse")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("heads_q,heads_k,dim", [(1, 1, 16), (4, 2, 32), (3, 1, 48), (8, 8, 64),
                                                 (6, 2, 80), (16, 4, 96), (5, 5, 112),
                                                 (16, 2, 128), (32, 1, 64)])
def test_one_token(dtype, bits, heads_q, heads_k, dim):
    c = Case(dtype, bits, heads_q, heads_k, dim, [1] * 7, [1, 0, 31, 32, 33, 300, 1500])
    c.check(*c.run())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("heads_q,heads_k,dim", [(2, 2, 16), (6, 2, 48), (4, 1, 64), (8, 2, 96),
                                                 (4, 4, 128)])
def test_some_tokens(dtype, bits, heads_q, heads_k, dim):
    """Drafted tokens, pieces of prompts, tokens without a key, whole documents."""
    c = Case(dtype, bits, heads_q, heads_k, dim, [3, 0, 17, 70, 1, 9, 5], [3, 4, 200, 70, 515, 6, 0])
    c.check(*c.run())
    c.check(*c.run(hints=(0, 0)))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("how", ["all", "prefix", "cap", "wide", "slopes", "all-slopes-cap"])
def test_masks_and_scores(dtype, bits, how):
    more = {"all": dict(causal=False), "prefix": dict(prefix=[40, 0, 9, 300]),
            "cap": dict(softcap=3.0), "wide": dict(softcap=200.0), "slopes": dict(slopes=True),
            "all-slopes-cap": dict(causal=False, slopes=True, softcap=20.0)}[how]
    for dim in (64, 128):
        c = Case(dtype, bits, 8, 4, dim, [20, 1, 9, 33], [100, 700, 9, 290], **more)
        c.check(*c.run())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("heads_q,heads_k,dim", [(4, 4, 32), (8, 2, 64), (12, 3, 96), (16, 2, 128)])
def test_shared_keys(dtype, bits, heads_q, heads_k, dim):
    # one prefix for some, another for others, none for the rest; one without keys
    c = Case(dtype, bits, heads_q, heads_k, dim, [1, 1, 2, 1, 30, 1, 1], [1, 90, 40, 5, 31, 0, 700],
             shared=[(0, 3, 333), (3, 2, 1), (5, 1, 0)])
    c.check(*c.run())
    c.check(*c.run(hints=(0, 0)))
    c = Case(dtype, bits, heads_q, heads_k, dim, [1] * 40, list(range(40)), shared=[(0, 40, 1200)])
    c.check(*c.run())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("own", [1, 9, 70])
@pytest.mark.parametrize("sharing", [1, 8, 70])
@pytest.mark.parametrize("softcap", [0.0, 5.0, 100.0])
def test_shared_and_own_keys_in_each_form(dtype, bits, dim, own, sharing, softcap):
    """16, 32 and 128 columns of either, causal, and rows that see no key at all."""
    many = max(sharing // own, 1)
    q_lens = [own] * many + [2, 3]
    k_lens = [own + 37 * i for i in range(many)] + [0, 1]
    c = Case(dtype, bits, 4, 1, dim, q_lens, k_lens, softcap=softcap,
             shared=[(0, many, 700), (many, 1, 0)])
    c.check(*c.run())


@pytest.mark.parametrize("hints", [(0, 0), (1, 1), (1, 100000), (5, 40), (1 << 30, 1 << 30)])
def test_hints_do_not_matter(hints):
    c = Case(torch.bfloat16, 8, 8, 2, 64, [40, 1, 7, 130], [2000, 900, 7, 131],
             shared=[(1, 2, 640)])
    c.check(*c.run(hints=hints))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("k_len", [1, 2, 3, 29, 30, 31, 32, 61, 130])
def test_the_end_of_the_cache(bits, head_major, k_len):
    """The last document ends with the arrays: nothing behind them is read."""
    for hk, dim in ((1, 16), (2, 128)):
        c = Case(torch.float16, bits, 4, hk, dim, [1], [k_len], head_major=head_major, tight=True)
        c.check(*c.run())


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", HALF)
def test_what_is_not_seen_does_not_matter(dtype, bits):
    c = Case(dtype, bits, 4, 2, 64, [5, 3, 40], [40, 3, 40], gap=5, prefix=[2, 0, 0])
    want = c.run()
    # rows between documents, and keys that only later tokens see
    for t in (c.k.low, c.k.step, c.v.low, c.v.step):
        keep = t.clone()
        t.fill_(NAN)
        for s, n in zip(c.k_starts, c.k_lens):
            t[:, s:s + n] = keep[:, s:s + n]
        t[:, c.k_starts[0] + 38:c.k_starts[0] + 40] = NAN   # the last two keys
        t[:, c.k_starts[2] + 20] = INF
    got = c.run()
    for d, (s, blind) in enumerate(zip(c.q_starts, ([0, 1, 2], [0, 1, 2], list(range(20))))):
        rows = [s + i for i in blind]
        assert torch.equal(got[0][rows], want[0][rows])
        assert torch.equal(got[1][:, rows], want[1][:, rows])
    # (a key of infinite numbers may get a score of -inf, and no weight)
    later = [c.q_starts[0] + 3, c.q_starts[0] + 4]
    assert torch.isnan(got[0][later]).all()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("bits", [8, 4])
def test_values_of_very_different_size(dtype, bits):
    """Steps from 2^-20 to 2^20 (bf16), growing along the keys."""
    spread = 12.0 if dtype == torch.bfloat16 else 4.0
    c = Case(dtype, bits, 2, 2, 32, [1, 2], [300, 500], spread=spread)
    c.check(*c.run())
    c = Case(dtype, bits, 2, 2, 32, [1, 2], [300, 500], spread=-spread)
    c.check(*c.run())


@pytest.mark.parametrize("size", [2.0 ** -20, 300.0])
def test_scores_far_apart(size):
    """Scores all but alike, and one key that takes all the weight."""
    c = Case(torch.bfloat16, 8, 4, 1, 64, [1, 1, 6], [400, 1100, 77])
    c.q *= size
    c.check(*c.run())
    c.scale = -c.scale
    c.cfg = raster.attention_config(c.dtype, 4, 1, 64, c.scale, True)
    c.check(*c.run())


def test_many_documents():
    c = Case(torch.bfloat16, 4, 4, 2, 32, [1] * 200, [(7 * i) % 90 for i in range(200)],
             shared=[(10 * i, 9, 20 + i) for i in range(19)])
    c.check(*c.run())
    c.check(*c.run(lse=False)[:1], None)


def test_long_cache():
    c = Case(torch.bfloat16, 8, 4, 1, 128, [1, 2], [70001, 40000], shared=[(0, 2, 30001)])
    c.check(*c.run())


def test_same_bits_on_a_stream_and_in_a_graph():
    c = Case(torch.float16, 4, 8, 2, 64, [1, 3, 1], [1000, 40, 7], shared=[(0, 2, 500)])
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    docs, shared = c.documents()
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    n = raster.gs_cached_attention_fwd_workspace_size(c.cfg, 4, docs, shared, c.rows_q, c.rows_k)
    space = torch.empty((n,), dtype=torch.uint8, device="cuda")
    args = (c.cfg, docs, shared, c.rows_q, c.rows_k, c.q, c.k.view(), c.v.view(), out, lse, space, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        raster.gs_cached_attention_fwd(*args)
    for i in range(4):
        c.q.copy_(_normal(90 + i, *c.q.shape))
        out.fill_(9.0)
        lse.fill_(9.0)
        space.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        fresh = c.run()
        used = slice(1, c.rows_q - 2)
        assert torch.equal(out[used], fresh[0][used]) and torch.equal(lse, fresh[1])
        c.check(out, lse)


def test_nothing_to_do():
    c = Case(torch.bfloat16, 8, 4, 2, 32, [], [])
    out, lse = c.run()
    assert (out == 9.0).all() and (lse == 9.0).all()
    # no cache at all: nothing is seen
    c = Case(torch.bfloat16, 8, 4, 2, 32, [1, 2], [0, 0])
    docs, _ = c.documents()
    out = torch.full((c.rows_q, 4, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    n = raster.gs_cached_attention_fwd_workspace_size(c.cfg, 8, docs, None, c.rows_q, 0)
    space = torch.empty((max(n, 256),), dtype=torch.uint8, device="cuda")
    none = Cache(0, 2, 32, 8).view()
    raster.gs_cached_attention_fwd(c.cfg, docs, None, c.rows_q, 0, c.q, none, none, out, None,
                                   space, n)
    assert (out[1:4] == 0).all() and (out[0] == 9.0).all() and (out[4:] == 9.0).all()
