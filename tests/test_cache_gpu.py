"""Caches of 8 and 4 bits: tokens written into them and read back, bit for bit
against 64 bits."""
import pytest
import torch

from differentiable_rasterization_amd import raster
from serving_util import Cache, head_codes, pack

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _normal(seed, dtype, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _copy(c):
    return [t.clone() for t in (c.codes, c.low, c.step)]


def _same(a, b):
    return all(torch.equal(torch.nan_to_num(x.double(), nan=-77.0),
                           torch.nan_to_num(y.double(), nan=-77.0)) for x, y in zip(a, b))


def _written(cache, x, tokens, rows):
    """What the cache holds after tokens went to rows."""
    codes, low, step = _copy(cache)
    u, lo, st = head_codes(x[tokens], cache.bits)
    codes[rows] = pack(u, cache.bits)
    low[:, rows], step[:, rows] = lo.T.float(), st.T.float()
    return [codes, low, step]


def _values(cache, rows, dtype):
    from serving_util import unpack
    u = unpack(cache.codes[rows], cache.bits).float()
    return (cache.low.T[rows][..., None] + cache.step.T[rows][..., None] * u).to(dtype)


# (q_start, q_len, k_start, k_len) of documents, rows of tokens and of the cache
LAYOUTS = [
    ([0], [1], [3], [1], 1, 4),
    ([0, 1, 2], [1, 1, 1], [40, 0, 20], [7, 12, 20], 3, 52),
    ([5, 0, 40, 41], [33, 5, 0, 17], [100, 0, 10, 40], [50, 5, 3, 17], 70, 150),
    ([0], [300], [0], [300], 300, 300),
    ([2, 10], [6, 20], [0, 8], [4, 20], 32, 30),             # two tokens without a key
    ([-3, 8, 30], [7, 100, 5], [-5, 60, 9], [9, 100, 5], 20, 64),  # outside: clamped
]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("heads,dim", [(1, 16), (3, 48), (8, 64), (2, 80), (5, 112), (4, 128)])
def test_write_and_read(dtype, bits, heads, dim):
    for case, (qs, ql, ks, kl, rows_q, rows_k) in enumerate(LAYOUTS):
        fused = _normal(case, dtype, rows_q, 3 * heads, dim)
        k, v = fused[:, heads:2 * heads], fused[:, 2 * heads:]
        caches = [Cache(rows_k, heads, dim, bits, head_major=bool(case & 1), spare=16 * (case & 2),
                        ld=rows_k + case) for _ in range(2)]
        tokens, rows, lost = [], [], []
        for a, n, b, m in zip(qs, ql, ks, kl):
            a0 = min(max(a, 0), rows_q)
            n = min(max(n, 0), rows_q - a0)
            b0 = min(max(b, 0), rows_k)
            m = min(max(m, 0), rows_k - b0)
            for i in range(n):
                if i + m - n >= 0:
                    tokens.append(a0 + i)
                    rows.append(b0 + i + m - n)
                else:
                    lost.append(a0 + i)
        want = [_written(c, x, tokens, rows) for c, x in zip(caches, (k, v))]
        docs = raster.documents(*map(_ints, (qs, ql, ks, kl)), max_q_len=case % 3)
        cfg = raster.cache_config(dtype, heads, dim)
        raster.gs_cache_write(cfg, docs, rows_q, rows_k, k, v, *[c.view() for c in caches])
        for c, w in zip(caches, want):
            assert _same(_copy(c), w)
        out = [torch.full((rows_q, heads + 2, dim), 9.0, dtype=dtype, device="cuda")
               for _ in range(2)]
        raster.gs_cache_read(cfg, docs, rows_q, rows_k, *[c.view() for c in caches],
                             *[t[:, 1:heads + 1] for t in out])
        for c, t in zip(caches, out):
            full = torch.full_like(t, 9.0)
            full[tokens, 1:heads + 1] = _values(c, rows, dtype)
            full[lost, 1:heads + 1] = 0.0
            assert torch.equal(t, full)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [32, 128])
def test_heads_without_codes(dtype, bits, dim):
    x = _normal(1, dtype, 10, 2, dim)
    x[0, 0], x[1, 1, 3], x[2, 0, 4], x[3, 1, dim - 1] = 2.5, NAN, INF, -INF
    x[4, 0] = 0.0
    x[4, 0, 1] = 2.0 ** -118 if dtype != torch.float16 else 2.0 ** -24
    x[5, 0] = 0.0
    x[5, 0, 9] = 2.0 ** -115 if dtype != torch.float16 else 65504.0
    x[6, 1, 0], x[6, 1, 1] = torch.finfo(dtype).max, -torch.finfo(dtype).max
    x[7], x[8, 0, 0], x[8, 0, 1] = NAN, INF, -INF
    # ties: codes half way between two
    x[9, 0] = 0.0
    x[9, 0, 0] = 2.0 ** bits - 1
    x[9, 0, 1:6] = torch.tensor([0.5, 1.5, 2.5, 6.5, 13.5], device="cuda").to(dtype)
    caches = [Cache(10, 2, dim, bits) for _ in range(2)]
    want = [_written(c, x, list(range(10)), list(range(10))) for c in caches]
    docs = raster.documents(_ints([0]), _ints([10]))
    cfg = raster.cache_config(dtype, 2, dim)
    raster.gs_cache_write(cfg, docs, 10, 10, x, x, *[c.view() for c in caches])
    assert all(_same(_copy(c), w) for c, w in zip(caches, want))
    out = [torch.empty_like(x) for _ in range(2)]
    raster.gs_cache_read(cfg, docs, 10, 10, *[c.view() for c in caches], *out)
    for c, t in zip(caches, out):
        assert _same([t], [_values(c, list(range(10)), dtype)])


def test_many_documents_and_a_graph():
    """300 requests of one token each, step after step, captured."""
    n, heads, dim, room = 300, 4, 64, 9
    cfg = raster.cache_config(torch.bfloat16, heads, dim)
    caches = [Cache(n * room, heads, dim, 8) for _ in range(2)]
    views = [c.view() for c in caches]
    kl = torch.ones(n, dtype=torch.int32, device="cuda")
    order = torch.randperm(n, device="cuda").int()
    docs = raster.documents(order, torch.ones_like(kl), torch.arange(n, device="cuda").int() * room,
                            kl, max_q_len=1)
    k, v = (torch.zeros((n, heads, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = [torch.zeros_like(k) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    raster.gs_cache_write(cfg, docs, n, n * room, k, v, *views, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        raster.gs_cache_write(cfg, docs, n, n * room, k, v, *views)
        raster.gs_cache_read(cfg, docs, n, n * room, *views, *out)
    for step in range(5):
        k.copy_(_normal(2 * step, torch.bfloat16, n, heads, dim))
        v.copy_(_normal(2 * step + 1, torch.bfloat16, n, heads, dim))
        kl.fill_(step + 1)
        rows = torch.arange(n, device="cuda") * room + step
        want = [_written(c, x, order.long(), rows) for c, x in zip(caches, (k, v))]
        graph.replay()
        torch.cuda.synchronize()
        for c, w, t in zip(caches, want, out):
            assert _same(_copy(c), w)
            full = torch.empty_like(t)
            full[order.long()] = _values(c, rows, torch.bfloat16)
            assert torch.equal(t, full)


def test_nothing_to_do():
    cfg = raster.cache_config(torch.float16, 2, 32)
    c = Cache(4, 2, 32, 4)
    before = _copy(c)
    none = torch.empty((0, 2, 32), dtype=torch.float16, device="cuda")
    empty = raster.documents(_ints([]), _ints([]))
    raster.gs_cache_write(cfg, empty, 0, 4, none, none, c.view(), Cache(4, 2, 32, 4).view())
    x = torch.full((3, 2, 32), 7.0, dtype=torch.float16, device="cuda")
    nothing = raster.documents(_ints([0]), _ints([0]), _ints([0]), _ints([0]))
    raster.gs_cache_write(cfg, nothing, 3, 4, x, x, c.view(), Cache(4, 2, 32, 4).view())
    assert _same(before, _copy(c))
    y = x.clone()
    raster.gs_cache_read(cfg, nothing, 3, 4, c.view(), Cache(4, 2, 32, 4).view(), x, y)
    assert (x == 7.0).all() and (y == 7.0).all()


@pytest.mark.parametrize("hint", [0, 1, 5, 8, 9, 100])
def test_hints_do_not_matter(hint):
    """Documents of one token, of some and of many, whatever the caller says of them."""
    ql, kl = [1, 0, 30, 8, 9], [4, 2, 33, 8, 10]
    qs, ks = [0, 1, 1, 31, 39], [0, 4, 6, 40, 50]
    x = _normal(hint, torch.float16, 48, 6, 48)
    k, v = x[:, :3], x[:, 3:]
    caches = [Cache(64, 3, 48, 4) for _ in range(2)]
    tokens = [a + i for a, n in zip(qs, ql) for i in range(n)]
    rows = [b + m - n + i for b, m, n in zip(ks, kl, ql) for i in range(n)]
    want = [_written(c, t, tokens, rows) for c, t in zip(caches, (k, v))]
    docs = raster.documents(*map(_ints, (qs, ql, ks, kl)), max_q_len=hint)
    cfg = raster.cache_config(torch.float16, 3, 48)
    raster.gs_cache_write(cfg, docs, 48, 64, k, v, *[c.view() for c in caches])
    assert all(_same(_copy(c), w) for c, w in zip(caches, want))
    out = [torch.full((48, 3, 48), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    raster.gs_cache_read(cfg, docs, 48, 64, *[c.view() for c in caches], *out)
    for c, t in zip(caches, out):
        assert torch.equal(t[tokens], _values(c, rows, torch.float16))
