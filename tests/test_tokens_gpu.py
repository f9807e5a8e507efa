"""The token operators' kernels against their 64-bit forms (token_util), at
the sizes and masks where they can go wrong.  The tolerances are token_util's
bounds of the kernels' roundings."""
import pytest
import torch

import token_util as tu
from differentiable_rasterization_amd import raster

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _space(nbytes):
    return torch.full((max(int(nbytes), 256),), 0xAB, dtype=torch.uint8, device="cuda")


def _view(gen, dtype, rows, heads, dim, layout, fill=None):
    """A [rows, heads, dim] tensor in one of three layouts."""
    if layout == "rows":
        t = torch.empty((rows, heads, dim), dtype=dtype, device="cuda")
    elif layout == "heads":
        t = torch.empty((heads, rows, dim), dtype=dtype, device="cuda").permute(1, 0, 2)
    else:  # columns of a wider projection, one head apart
        t = torch.empty((rows, heads + 3, dim + 8), dtype=dtype,
                        device="cuda")[:, 1:heads + 1, :dim]
    t.copy_(_normal(gen, dtype, rows, heads, dim) if fill is None else
            torch.full((rows, heads, dim), fill, dtype=dtype, device="cuda"))
    return t


# ---------------------------------------------------------------------------
# Norm and rotary position
# ---------------------------------------------------------------------------
QK = [
    # rows, heads_q, heads_k, dim, rotary, interleaved, norm, layout
    (1, 1, 1, 8, 0, False, True, "rows"),
    (1, 4, 2, 64, 64, False, True, "rows"),
    (3, 5, 3, 24, 16, False, True, "fused"),
    (7, 3, 1, 96, 48, False, True, "heads"),
    (65, 6, 2, 128, 128, True, True, "fused"),
    (130, 2, 2, 40, 32, True, False, "rows"),
    (33, 2, 1, 512, 256, False, True, "rows"),
    (17, 1, 2, 264, 64, False, True, "rows"),
    (2000, 9, 3, 128, 64, False, True, "fused"),
    (5001, 4, 4, 64, 64, True, True, "rows"),
]


@pytest.mark.parametrize("dtype", [torch.float32] + TYPES)
@pytest.mark.parametrize("case", QK)
def test_qk_norm_rope(case, dtype):
    rows, hq, hk, dim, rotary, inter, norm, layout = case
    gen = _gen(rows + dim)
    q, k = (_view(gen, dtype, rows, h, dim, layout) for h in (hq, hk))
    dyq, dyk = (_view(gen, dtype, rows, h, dim, layout) for h in (hq, hk))
    pos = torch.randint(0, 100000, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    freq = torch.rand(max(rotary // 2, 1), generator=gen, device="cuda")
    wq, wk = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda") for _ in range(2))
    eps, amp = 1e-6, 1.25
    cfg = raster.qk_config(dtype, hq, hk, dim, rotary, inter, norm, eps, amp)
    oq, ok = (_view(gen, dtype, rows, h, dim, layout, 7.0) for h in (hq, hk))
    dq, dk = (_view(gen, dtype, rows, h, dim, layout, 7.0) for h in (hq, hk))
    dwq, dwk = (torch.full((dim,), 7.0, device="cuda") for _ in range(2))
    raster.gs_qk_norm_rope_fwd(cfg, rows, pos, freq, wq, wk, q, k, oq, ok)
    n = raster.gs_qk_norm_rope_bwd_workspace_size(cfg, rows)
    raster.gs_qk_norm_rope_bwd(cfg, rows, pos, freq, wq, wk, q, k, dyq, dyk, dq, dk, dwq, dwk,
                               _space(n), n)
    turn = tu.turn_matrix(pos, freq, dim, rotary, inter, amp)
    u = tu.U[dtype]
    # fp32 of a sum of dim squares, a root, three products and the angle: 4e-6
    for x, w, y, dy, dx, dw in ((q, wq, oq, dyq, dq, dwq), (k, wk, ok, dyk, dk, dwk)):
        w = w if norm else None
        want, size = tu.qk_forward(x, w, turn, eps)
        tu.close(y, want, u * want.abs() + 4e-6 * size + tu.TINY[dtype], "y")
        gx, agx, gw, agw = tu.qk_backward(x, w, turn, eps, dy)
        tu.close(dx, gx, u * gx.abs() + 8e-6 * agx + tu.TINY[dtype], "dx")
        if norm:
            # a sum of some hundred fp32 additions a level
            tu.close(dw, gw, 3e-5 * agw, "dw")
        else:
            assert (dw == 7.0).all()


def test_qk_in_place_and_repeatable():
    gen = _gen(1)
    rows, hq, hk, dim = 300, 6, 2, 96
    q, k = (_normal(gen, torch.bfloat16, rows, h, dim) for h in (hq, hk))
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    freq = torch.rand(24, generator=gen, device="cuda")
    w = torch.ones(dim, device="cuda")
    cfg = raster.qk_config(torch.bfloat16, hq, hk, dim, 48)
    a, b = torch.empty_like(q), torch.empty_like(k)
    raster.gs_qk_norm_rope_fwd(cfg, rows, pos, freq, w, w, q, k, a, b)
    q2, k2 = q.clone(), k.clone()
    raster.gs_qk_norm_rope_fwd(cfg, rows, pos, freq, w, w, q2, k2, q2, k2)
    assert torch.equal(a, q2) and torch.equal(b, k2)


def test_qk_bad_token_stays_alone():
    gen = _gen(2)
    q, k = (_normal(gen, torch.float32, 9, h, 64) for h in (4, 2))
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    freq, w = torch.rand(32, generator=gen, device="cuda"), torch.ones(64, device="cuda")
    cfg = raster.qk_config(torch.float32, 4, 2, 64)
    clean = [torch.empty_like(q), torch.empty_like(k)]
    raster.gs_qk_norm_rope_fwd(cfg, 9, pos, freq, w, w, q, k, *clean)
    q[4, 1, 3], k[5, 0, 0] = float("nan"), float("inf")
    got = [torch.empty_like(q), torch.empty_like(k)]
    raster.gs_qk_norm_rope_fwd(cfg, 9, pos, freq, w, w, q, k, *got)
    for a, b, (r, h) in ((clean[0], got[0], (4, 1)), (clean[1], got[1], (5, 0))):
        assert not torch.isfinite(b[r, h]).all()
        a[r, h] = b[r, h] = 0.0
        assert torch.equal(a, b)


def test_qk_no_rows_and_zero_rows():
    cfg = raster.qk_config(torch.float32, 2, 1, 32)
    w, dw = torch.ones(32, device="cuda"), [torch.full((32,), 3.0, device="cuda") for _ in "qk"]
    raster.gs_qk_norm_rope_fwd(cfg, 0, None, None, None, None, None, None, None, None)
    raster.gs_qk_norm_rope_bwd(cfg, 0, None, None, None, None, None, None, None, None, None, None,
                               *dw, None, 0)
    assert all((t == 0).all() for t in dw)
    # a row of zeros: eps keeps it at zero
    x, k = torch.zeros((1, 2, 32), device="cuda"), torch.zeros((1, 1, 32), device="cuda")
    pos, freq = _ints([5]), torch.ones(16, device="cuda")
    raster.gs_qk_norm_rope_fwd(cfg, 1, pos, freq, w, w, x, k, x, k)
    assert (x == 0).all() and (k == 0).all()


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
ATTENTION = [
    # lengths of queries, of keys (None: the same), heads_q, heads_k, dim, options
    ([1], None, 1, 1, 8, {}),
    ([1, 0, 3], None, 2, 1, 16, dict(causal=True)),
    ([64], None, 2, 2, 64, dict(causal=True)),
    ([65, 63, 128, 127, 129], None, 4, 2, 64, dict(causal=True)),
    ([65, 63, 128, 127, 129], None, 3, 1, 128, dict(causal=False)),
    ([200, 1, 31, 33], None, 6, 2, 96, dict(causal=True, softcap=4.0)),
    ([97, 130], None, 4, 4, 40, dict(causal=True, slopes=True)),
    ([97, 130], None, 4, 1, 72, dict(causal=False, slopes=True, softcap=20.0)),
    ([150, 77], None, 2, 2, 128, dict(causal=True, prefix=[70, 100])),
    ([150, 77, 5], None, 8, 2, 64, dict(causal=True, prefix=[149, 0, 9], slopes=True)),
    # more keys than tokens (a cache), fewer (rows that see nothing), none
    ([1, 1, 1], [300, 1, 64], 8, 2, 128, dict(causal=True)),
    ([1, 2, 4], [1000, 513, 77], 5, 5, 64, dict(causal=True, slopes=True)),
    ([40, 100, 7], [10, 1, 0], 2, 1, 64, dict(causal=True)),
    ([40, 100, 7], [10, 1, 0], 2, 1, 64, dict(causal=False, softcap=10.0)),
    ([50], [20], 2, 2, 32, dict(causal=True, prefix=[8])),
    ([700], None, 16, 2, 128, dict(causal=True, softcap=30.0)),
    ([3], [2500], 12, 2, 128, dict(causal=True)),
    ([33], [4000], 1, 1, 64, dict(causal=False)),
]


def _attention_reference(case, q, k, v, do, qs, ks, scale, slopes, dtype):
    lq, lk, hq, hk, dim, opt = case
    lk = lq if lk is None else lk
    g = hq // hk
    ref = {n: torch.zeros(t.shape, dtype=torch.float64, device="cuda")
           for n, t in (("o", q), ("eo", q), ("dq", q), ("edq", q), ("dk", k), ("edk", k),
                        ("dv", v), ("edv", v))}
    ref["lse"] = torch.full((hq, q.shape[0]), float("nan"), dtype=torch.float64, device="cuda")
    prefix = opt.get("prefix", [0] * len(lq))
    u = tu.U[dtype]
    for d in range(len(lq)):
        a, b = slice(qs[d], qs[d] + lq[d]), slice(ks[d], ks[d] + lk[d])
        seen, away = tu.seen_and_away(lq[d], lk[d], opt.get("causal", False), prefix[d], "cuda")
        for h in range(hq):
            x, y, z, w = (t.double() for t in (q[a, h], k[b, h // g], v[b, h // g], do[a, h]))
            r = tu.attention_head(x, y, z, w, scale, opt.get("softcap", 0.0),
                                  float(slopes[h]) if slopes is not None else 0.0, seen, away)
            ref["o"][a, h], ref["lse"][h, a] = r["o"], r["lse"]
            tiny = tu.TINY[dtype] * (r["p"] > 0).double() @ z.abs()
            ref["eo"][a, h] = u * r["o"].abs() + (u + tu.EPS32) * r["ao"] + tiny
            eq, ek, ev = tu.attention_error(r, x, y, z, w, scale, dtype)
            ref["dq"][a, h], ref["edq"][a, h] = r["dq"], eq + u * r["dq"].abs()
            ref["dk"][b, h // g] += r["dk"]
            ref["dv"][b, h // g] += r["dv"]
            ref["edk"][b, h // g] += ek
            ref["edv"][b, h // g] += ev
    for n in ("dk", "dv"):
        ref["e" + n] += u * ref[n].abs()
    return ref


def _run_attention(case, dtype, layout, seed=0, gap=3, bounds=True, stream=None):
    lq, lk, hq, hk, dim, opt = case
    gen = _gen(seed + 17 * len(lq) + dim)
    qs, rows_q = tu.starts_of(lq, gap)
    if lk is None:
        ks, rows_k = qs, rows_q
    else:
        # keys of the documents stand in the opposite order
        s, rows_k = tu.starts_of(lk[::-1], gap)
        ks = s[::-1]
    q = _view(gen, dtype, rows_q, hq, dim, layout)
    k, v = (_view(gen, dtype, rows_k, hk, dim, layout) for _ in range(2))
    do = _view(gen, dtype, rows_q, hq, dim, layout)
    klen = lq if lk is None else lk
    for t, st, ln in ((q, qs, lq), (do, qs, lq), (k, ks, klen), (v, ks, klen)):
        # what stands between the documents does not matter
        used = torch.zeros(t.shape[0], dtype=torch.bool, device="cuda")
        for a, n in zip(st, ln):
            used[a:a + n] = True
        t[~used] = float("nan")
    slopes = None
    if opt.get("slopes"):
        slopes = torch.linspace(0.02, 0.5, hq, device="cuda")
    scale = tu.sqrt_scale(dim)
    cfg = raster.attention_config(dtype, hq, hk, dim, scale, opt.get("causal", False),
                                  opt.get("softcap", 0.0), slopes)
    docs = raster.documents(_ints(qs), _ints(lq), None if lk is None else _ints(ks),
                            None if lk is None else _ints(lk),
                            _ints(opt["prefix"]) if "prefix" in opt else None,
                            max_q_len=max(lq) if bounds else 0,
                            max_k_len=max(klen) if bounds else 0)
    o = _view(gen, dtype, rows_q, hq, dim, layout, 7.0)
    lse = torch.full((hq, rows_q), 7.0, device="cuda")
    dq = _view(gen, dtype, rows_q, hq, dim, layout, 7.0)
    dk, dv = (_view(gen, dtype, rows_k, hk, dim, layout, 7.0) for _ in range(2))
    nf = raster.gs_attention_fwd_workspace_size(cfg, docs, rows_q, rows_k)
    nb = raster.gs_attention_bwd_workspace_size(cfg, docs, rows_q, rows_k)
    ws = _space(max(nf, nb))
    raster.gs_attention_fwd(cfg, docs, rows_q, rows_k, q, k, v, o, lse, ws, nf, stream)
    raster.gs_attention_bwd(cfg, docs, rows_q, rows_k, q, k, v, o, lse, do, dq, dk, dv, ws, nb,
                            stream)
    # and without the logarithms, as in serving
    o2 = _view(gen, dtype, rows_q, hq, dim, layout, 7.0)
    raster.gs_attention_fwd(cfg, docs, rows_q, rows_k, q, k, v, o2, None, ws, nf, stream)
    return dict(q=q, k=k, v=v, do=do, o=o, o2=o2, lse=lse, dq=dq, dk=dk, dv=dv, qs=qs, ks=ks,
                scale=scale, slopes=slopes)


@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", ATTENTION, ids=range(len(ATTENTION)))
def test_attention(case, dtype, layout):
    _check_attention(case, dtype, layout)


def _check_attention(case, dtype, layout):
    r = _run_attention(case, dtype, layout, bounds=layout != "heads")
    lq, lk, hq, hk, dim, opt = case
    klen = lq if lk is None else lk
    ref = _attention_reference(case, r["q"], r["k"], r["v"], r["do"], r["qs"], r["ks"],
                               r["scale"], r["slopes"], dtype)
    inside = torch.zeros(r["q"].shape[0], dtype=torch.bool, device="cuda")
    for a, n in zip(r["qs"], lq):
        inside[a:a + n] = True
    kin = torch.zeros(r["k"].shape[0], dtype=torch.bool, device="cuda")
    for a, n in zip(r["ks"], klen):
        kin[a:a + n] = True
    tu.close(r["o"][inside], ref["o"][inside], ref["eo"][inside], "o")
    assert torch.equal(r["o"], r["o2"])
    got, want = r["lse"][:, inside].double(), ref["lse"][:, inside]
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    fin = torch.isfinite(want)
    tu.close(got[fin], want[fin], 1e-6 * want[fin].abs() + tu.EPS32, "lse")
    for n, at in (("dq", inside), ("dk", kin), ("dv", kin)):
        tu.close(r[n][at], ref[n][at], ref["e" + n][at], n)
    # rows of no document are not written
    for n, at in (("o", inside), ("dq", inside), ("dk", kin), ("dv", kin)):
        assert (r[n][~at] == 7.0).all(), n
    assert (r["lse"][:, ~inside] == 7.0).all()


# many heads: enough workgroups for the forms with 128 columns or keys each
MANY = [
    ([130, 65, 257, 1], None, 128, 64, 64, dict(causal=True)),
    ([130, 65, 257, 1], None, 64, 64, 128, dict(causal=True)),
    ([200, 64, 100], None, 128, 32, 128, dict(causal=True, softcap=8.0, prefix=[30, 64, 0])),
    ([200, 64, 100], None, 128, 128, 40, dict(causal=True, slopes=True)),
    ([150, 200], [400, 70], 128, 64, 96, dict(causal=True, slopes=True, softcap=15.0)),
    ([150, 200, 9], [400, 70, 0], 128, 64, 128, dict(causal=False)),
    ([3] * 150 + [0, 1, 65], None, 4, 2, 32, dict(causal=True)),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case", MANY, ids=range(len(MANY)))
def test_attention_many_heads_or_documents(case, dtype):
    _check_attention(case, dtype, "fused")


def _captured(run, outputs):
    """Replays of a captured call against its eager results, with the
    program's own work in between."""
    run()
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for t in outputs:
            t.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w)


def test_token_calls_can_be_captured():
    gen = _gen(21)
    n, hq, hk, dim, dtype = 300, 8, 2, 64, torch.bfloat16
    q, k, v, do = (_normal(gen, dtype, n, h, dim) for h in (hq, hk, hk, hq))
    o, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    lse = torch.empty((hq, n), device="cuda")
    cfg = raster.attention_config(dtype, hq, hk, dim, 0.125, True)
    docs = raster.documents(_ints([0, 100]), _ints([100, 200]))
    nb = max(raster.gs_attention_fwd_workspace_size(cfg, docs, n, n),
             raster.gs_attention_bwd_workspace_size(cfg, docs, n, n))
    ws = _space(nb)

    def attention():
        raster.gs_attention_fwd(cfg, docs, n, n, q, k, v, o, lse, ws, nb)
        raster.gs_attention_bwd(cfg, docs, n, n, q, k, v, o, lse, do, dq, dk, dv, ws, nb)
    _captured(attention, (o, lse, dq, dk, dv))

    # one token over long caches: split over the keys and joined
    one = raster.documents(_ints([0, 1]), _ints([1, 1]), _ints([0, 4096]), _ints([4000, 1500]),
                           max_q_len=1, max_k_len=4000)
    ck, cv = (_normal(gen, dtype, 8192, hk, dim) for _ in range(2))
    oo = torch.empty_like(q[:2])
    ns = raster.gs_attention_fwd_workspace_size(cfg, one, 2, 8192)
    assert ns > 0
    wss = _space(ns)
    _captured(lambda: raster.gs_attention_fwd(cfg, one, 2, 8192, q[:2], ck, cv, oo, None, wss, ns),
              (oo,))

    ch = 64
    gate, x, dy = (_normal(gen, dtype, n, ch) for _ in range(3))
    y, df, dx = (torch.empty_like(x) for _ in range(3))
    end, ds = torch.zeros((2, ch), device="cuda"), torch.zeros((2, ch), device="cuda")
    scan = raster.scan_config(dtype, ch)
    saved = _space(raster.gs_gated_scan_saved_size(scan, docs, n))
    nc = raster.gs_gated_scan_fwd_workspace_size(scan, docs, n)
    wsc = _space(nc)

    def gated():
        raster.gs_gated_scan_fwd(scan, docs, n, gate, x, None, y, end, saved, wsc, nc)
        raster.gs_gated_scan_bwd(scan, docs, n, gate, x, saved, dy, None, df, dx, ds, wsc, nc)
    _captured(gated, (y, end, df, dx, ds))

    qk = raster.qk_config(dtype, hq, hk, dim)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freq, w = torch.rand(32, generator=gen, device="cuda"), torch.ones(dim, device="cuda")
    dwq, dwk = torch.empty_like(w), torch.empty_like(w)
    nq = raster.gs_qk_norm_rope_bwd_workspace_size(qk, n)
    wsq = _space(nq)

    def turned():
        raster.gs_qk_norm_rope_fwd(qk, n, pos, freq, w, w, q, k, dq, dk)
        raster.gs_qk_norm_rope_bwd(qk, n, pos, freq, w, w, q, k, do, v, o, dv, dwq, dwk, wsq, nq)
    _captured(turned, (dq, dk, o, dv, dwq, dwk))


@pytest.mark.parametrize("case", [ATTENTION[3], ATTENTION[9], ATTENTION[11], ATTENTION[16]])
def test_attention_repeats_bit_for_bit_and_on_another_stream(case):
    a = _run_attention(case, torch.bfloat16, "rows")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _run_attention(case, torch.bfloat16, "rows")
    side.synchronize()
    for n in ("o", "lse", "dq", "dk", "dv"):
        x, y = a[n], b[n]
        same = (x == y) | (torch.isnan(x) & torch.isnan(y))
        assert same.all(), n


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_bad_document_stays_alone(bad):
    """A document of non-finite values next to others inside the same tiles."""
    gen = _gen(5)
    lens, hq, hk, dim, dtype = [20, 30, 25], 4, 2, 64, torch.bfloat16
    qs, rows = tu.starts_of(lens)
    q, k, v, do = (_normal(gen, dtype, rows, h, dim) for h in (hq, hk, hk, hq))
    cfg = raster.attention_config(dtype, hq, hk, dim, 0.125, True)
    docs = raster.documents(_ints(qs), _ints(lens))
    def run():
        o, dq = torch.zeros_like(q), torch.zeros_like(q)
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        lse = torch.zeros((hq, rows), device="cuda")
        nf = raster.gs_attention_fwd_workspace_size(cfg, docs, rows, rows)
        nb = raster.gs_attention_bwd_workspace_size(cfg, docs, rows, rows)
        ws = _space(max(nf, nb))
        raster.gs_attention_fwd(cfg, docs, rows, rows, q, k, v, o, lse, ws, nf)
        raster.gs_attention_bwd(cfg, docs, rows, rows, q, k, v, o, lse, do, dq, dk, dv, ws, nb)
        return o, dq, dk, dv
    clean = run()
    for t in (q, k, v, do):
        t[20:50] = bad
    dirty = run()
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[20:50] = False
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])


def test_attention_far_rows_pass_32_bit_offsets():
    """Keys and values whose element offsets pass 2^32, in a cache of few used
    rows: the last document's keys stand at its end."""
    dtype, hq, hk, dim = torch.bfloat16, 4, 2, 128
    gen = _gen(9)
    rows_k = (1 << 32) // (hk * dim) + 5000
    k = torch.empty((rows_k, hk, dim), dtype=dtype, device="cuda")
    v = torch.empty((rows_k, hk, dim), dtype=dtype, device="cuda")
    starts, lens = [7, rows_k - 700], [130, 700]
    for s, n in zip(starts, lens):
        k[s:s + n] = _normal(gen, dtype, n, hk, dim)
        v[s:s + n] = _normal(gen, dtype, n, hk, dim)
    q = _normal(gen, dtype, 2, hq, dim)
    cfg = raster.attention_config(dtype, hq, hk, dim, tu.sqrt_scale(dim), True)
    docs = raster.documents(_ints([0, 1]), _ints([1, 1]), _ints(starts), _ints(lens),
                            max_q_len=1, max_k_len=700)
    o = torch.zeros_like(q)
    n = raster.gs_attention_fwd_workspace_size(cfg, docs, 2, rows_k)
    raster.gs_attention_fwd(cfg, docs, 2, rows_k, q, k, v, o, None, _space(n), n)
    for d, (s, ln) in enumerate(zip(starts, lens)):
        seen, away = tu.seen_and_away(1, ln, True, 0, "cuda")
        for h in range(hq):
            r = tu.attention_head(q[d:d + 1, h].double(), k[s:s + ln, h // 2].double(),
                                  v[s:s + ln, h // 2].double(), None, tu.sqrt_scale(dim), 0.0,
                                  0.0, seen, away)
            u = tu.U[dtype]
            tu.close(o[d:d + 1, h], r["o"], u * r["o"].abs() + (u + tu.EPS32) * r["ao"], "o")


def test_attention_ranges_are_clamped():
    """Starts and lengths that leave the buffers are cut to them."""
    gen = _gen(3)
    q, k, v = (_normal(gen, torch.float16, 50, 2, 64) for _ in range(3))
    cfg = raster.attention_config(torch.float16, 2, 2, 64, 0.1)
    outs = []
    for start, length in (([10], [40]), ([10], [1000000])):
        docs = raster.documents(_ints(start), _ints(length))
        o = torch.zeros_like(q)
        n = raster.gs_attention_fwd_workspace_size(cfg, docs, 50, 50)
        raster.gs_attention_fwd(cfg, docs, 50, 50, q, k, v, o, None, _space(n), n)
        outs.append(o)
    assert torch.equal(*outs) and (outs[0][:10] == 0).all() and (outs[0][10:] != 0).any()


def test_attention_gradient_against_differences():
    """The kernels' gradients along random directions against central
    differences of the 64-bit forward."""
    case = ([60, 33], None, 4, 2, 64, dict(causal=True, prefix=[20, 0], softcap=8.0, slopes=True))
    dtype = torch.float16
    r = _run_attention(case, dtype, "rows", gap=0)
    lq, _, hq, hk, dim, opt = case

    def loss(q, k, v):
        total = 0.0
        for d in range(len(lq)):
            a = slice(r["qs"][d], r["qs"][d] + lq[d])
            seen, away = tu.seen_and_away(lq[d], lq[d], True, opt["prefix"][d], "cuda")
            for h in range(hq):
                o = tu.attention_head(q[a, h], k[a, h // 2], v[a, h // 2], None, r["scale"], 8.0,
                                      float(r["slopes"][h]), seen, away)["o"]
                total += float((o * r["do"][a, h].double()).sum())
        return total
    ref = _attention_reference(case, r["q"], r["k"], r["v"], r["do"], r["qs"], r["ks"],
                               r["scale"], r["slopes"], dtype)
    base = [r[n].double() for n in "qkv"]
    gen = _gen(77)
    for i, n in enumerate("qkv"):
        d = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - 1e-4 * d, base[i] + 1e-4 * d
        want = (loss(*hi) - loss(*lo)) / 2e-4
        have = float((r["d" + n].double() * d).sum())
        # independent errors of the elements along a random direction: their
        # root sum of squares, six times
        tol = 6.0 * float(((ref["ed" + n] * d) ** 2).sum().sqrt()) + 1e-4
        assert abs(have - want) <= tol, (n, have, want, tol)


def test_attention_nothing_to_do():
    cfg = raster.attention_config(torch.float16, 2, 2, 64, 0.1)
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    docs = raster.documents(empty, empty)
    raster.gs_attention_fwd(cfg, docs, 0, 0, None, None, None, None, None, None, 0)
    raster.gs_attention_bwd(cfg, docs, 0, 0, *([None] * 4), None, *([None] * 4), None, 0)
    # tokens without any key at all
    q = torch.ones((4, 2, 64), dtype=torch.float16, device="cuda")
    o, dq = torch.ones_like(q), torch.ones_like(q)
    docs = raster.documents(_ints([0]), _ints([4]), _ints([0]), _ints([0]))
    lse = torch.zeros((2, 4), device="cuda")
    n = raster.gs_attention_fwd_workspace_size(cfg, docs, 4, 0)
    raster.gs_attention_fwd(cfg, docs, 4, 0, q, None, None, o, lse, _space(n), n)
    n = raster.gs_attention_bwd_workspace_size(cfg, docs, 4, 0)
    raster.gs_attention_bwd(cfg, docs, 4, 0, q, None, None, o, lse, q.clone(), dq, None, None,
                            _space(n), n)
    assert (o == 0).all() and (dq == 0).all() and (lse == -float("inf")).all()


# ---------------------------------------------------------------------------
# Gated scan
# ---------------------------------------------------------------------------
SCAN = [
    # lengths, channels, coupled
    ([1], 8, True),
    ([1, 1, 0, 1], 24, False),
    ([5, 64, 17], 264, True),
    ([65], 128, False),
    ([63, 64, 65, 0, 128, 129, 1], 520, True),
    ([1000, 16, 15], 256, False),
    ([5000], 16, True),
]


def _run_scan(lens, channels, coupled, dtype, gap=2, states=True, bounds=True):
    gen = _gen(channels + sum(lens))
    starts, n = tu.starts_of(lens, gap)
    n = max(n, 1)
    fused = torch.randn((n, 2 * channels), generator=gen, device="cuda")
    fused[:, :channels] = fused[:, :channels] * 2 + 2
    used = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, m in zip(starts, lens):
        used[a:a + m] = True
    fused[~used] = float("nan")
    fused = fused.to(dtype)
    gate, x = fused[:, :channels], fused[:, channels:]
    dy = _normal(gen, dtype, n, channels)
    dy[~used] = float("nan")
    h0, dh = (torch.randn((len(lens), channels), generator=gen, device="cuda") for _ in range(2))
    docs = raster.documents(_ints(starts), _ints(lens), max_q_len=max(lens) if bounds else 0)
    cfg = raster.scan_config(dtype, channels, coupled)
    y, df, dx = (torch.full((n, channels), 7.0, dtype=dtype, device="cuda") for _ in range(3))
    ho, dho = (torch.full_like(h0, 7.0) for _ in range(2))
    saved = _space(raster.gs_gated_scan_saved_size(cfg, docs, n))
    nf = raster.gs_gated_scan_fwd_workspace_size(cfg, docs, n)
    nb = raster.gs_gated_scan_bwd_workspace_size(cfg, docs, n)
    ws = _space(max(nf, nb))
    raster.gs_gated_scan_fwd(cfg, docs, n, gate, x, h0 if states else None, y, ho, saved, ws, nf)
    raster.gs_gated_scan_bwd(cfg, docs, n, gate, x, saved, dy, dh if states else None, df, dx,
                             dho, ws, nb)
    return dict(gate=gate, x=x, dy=dy, h0=h0, dh=dh, y=y, df=df, dx=dx, state=ho, dstate=dho,
                starts=starts, used=used, cfg=cfg, docs=docs, n=n)


@pytest.mark.parametrize("states", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32] + TYPES)
@pytest.mark.parametrize("case", SCAN, ids=range(len(SCAN)))
def test_gated_scan(case, dtype, states):
    lens, channels, coupled = case
    r = _run_scan(lens, channels, coupled, dtype, states=states, bounds=states)
    u = tu.U[dtype]
    zero = torch.zeros(channels, device="cuda")
    for d, (a, n) in enumerate(zip(r["starts"], lens)):
        at = slice(a, a + n)
        ref = tu.scan_document(r["gate"][at], r["x"][at], r["h0"][d] if states else zero, coupled,
                               r["dy"][at], r["dh"][d] if states else zero)
        for got, want, err in ((r["y"][at], ref["y"], ref["ey"]), (r["dx"][at], ref["dx"],
                               ref["edx"]), (r["df"][at], ref["df"], ref["edf"])):
            if n:
                tu.close(got, want, u * want.abs() + err + tu.TINY[dtype], "document %d" % d)
        tu.close(r["state"][d], ref["state"], ref["estate"] + 1e-30, "state %d" % d)
        tu.close(r["dstate"][d], ref["dstate"], ref["edstate"] + 1e-30, "dstate %d" % d)
    for t in ("y", "df", "dx"):
        assert (r[t][~r["used"]] == 7.0).all()


def test_gated_scan_carried_on_in_pieces():
    """A document in one call, and one token at a time with the state carried
    in place: the same outputs."""
    gen = _gen(11)
    n, ch = 90, 72
    gate, x = _normal(gen, torch.float32, n, ch), _normal(gen, torch.float32, n, ch)
    cfg = raster.scan_config(torch.float32, ch, True)
    whole, state = torch.empty_like(x), torch.zeros((1, ch), device="cuda")
    docs = raster.documents(_ints([0]), _ints([n]))
    nb = raster.gs_gated_scan_fwd_workspace_size(cfg, docs, n)
    end = torch.empty_like(state)
    raster.gs_gated_scan_fwd(cfg, docs, n, gate, x, state, whole, end, None, _space(nb), nb)
    one = raster.documents(_ints([0]), _ints([1]), max_q_len=1)
    steps = torch.empty_like(x)
    for t in range(n):
        raster.gs_gated_scan_fwd(cfg, one, 1, gate[t:t + 1], x[t:t + 1], state, steps[t:t + 1],
                                 state, None, None, 0)
    ref = tu.scan_document(gate, x, torch.zeros(ch, device="cuda"), True)
    tu.close(steps, ref["y"], ref["ey"] + 2.0 ** -24 * ref["y"].abs(), "steps")
    tu.close(whole, ref["y"], ref["ey"] + 2.0 ** -24 * ref["y"].abs(), "whole")
    tu.close(state[0], end[0], 2 * ref["estate"], "state")


def _recurrence(a, u, start):
    """h_t = a_t h_{t-1} + u_t down the rows, in 64 bits, by doubling."""
    a, h = a.double().clone(), u.double().clone()
    h[0] += a[0] * start.double()
    s = 1
    while s < len(h):
        h[s:] = h[s:] + a[s:] * h[:-s]
        a[s:] = a[s:] * a[:-s]
        s *= 2
    return h


def _after(h, start):
    return torch.cat([start.double()[None], h[:-1]])


def _scan_long(gate, x, h0, coupled, dy, dh):
    """tu.scan_document's values and bounds for documents of any length."""
    f, x, dy = gate.double(), x.double(), dy.double()
    a, z = torch.sigmoid(f), torch.sigmoid(-f)
    none = torch.zeros_like(a[0])
    u = z * x if coupled else x
    y = _recurrence(a, u, h0)
    before = _after(y, h0)
    ey = _recurrence(a, tu.GATE * (a * before.abs() + u.abs()), none)
    ebefore = _after(ey, none)
    later = torch.cat([a[1:], torch.ones_like(a[:1])]).flip(0)
    g = _recurrence(later, dy.flip(0), dh).flip(0)
    e = g - dy
    gnext = torch.cat([g[1:].abs(), none[None]])
    eg = _recurrence(later, (later.flip(0) * tu.GATE * gnext + tu.GATE
                             * (dy.abs() + e.abs())).flip(0), none).flip(0)
    d = before - x if coupled else before
    ad = before.abs() + (x.abs() if coupled else 0.0)
    w = z if coupled else 1.0
    return dict(y=y, ey=ey, state=y[-1], estate=ey[-1], dx=g * w, edx=(eg + tu.GATE * g.abs()) * w,
                df=g * d * a * z, dstate=a[0] * g[0], edstate=a[0] * (eg[0] + tu.GATE * g[0].abs()),
                edf=(eg * d.abs() + g.abs() * (ebefore + 2.0 * tu.GATE * ad)) * a * z)


def test_gated_scan_long_reference():
    gen = _gen(21)
    gate, x, dy = (_normal(gen, torch.float32, 77, 3) for _ in range(3))
    h0, dh = (torch.randn(3, generator=gen, device="cuda") for _ in range(2))
    for coupled in (True, False):
        a = tu.scan_document(gate, x, h0, coupled, dy, dh)
        b = _scan_long(gate, x, h0, coupled, dy, dh)
        for key, want in a.items():
            assert torch.allclose(b[key], want, rtol=1e-11, atol=1e-13), key


# a few chunks and a thousand of them; more tokens than a pass is made for
@pytest.mark.parametrize("dtype", [torch.float32] + TYPES)
@pytest.mark.parametrize("lens,channels,coupled", [
    ([700, 100000, 3], 136, True), ([262144], 8, False), ([262145, 300, 0, 64], 16, True)])
def test_gated_scan_long_documents(lens, channels, coupled, dtype):
    r = _run_scan(lens, channels, coupled, dtype)
    u = tu.U[dtype]
    for d, (a, n) in enumerate(zip(r["starts"], lens)):
        if n == 0:
            assert torch.equal(r["state"][d], r["h0"][d]) and torch.equal(r["dstate"][d], r["dh"][d])
            continue
        at = slice(a, a + n)
        ref = _scan_long(r["gate"][at], r["x"][at], r["h0"][d], coupled, r["dy"][at], r["dh"][d])
        for key in ("y", "dx", "df"):
            want = ref[key]
            tu.close(r[key][at], want, u * want.abs() + ref["e" + key] + tu.TINY[dtype], key)
        tu.close(r["state"][d], ref["state"], ref["estate"] + 1e-30, "state")
        tu.close(r["dstate"][d], ref["dstate"], ref["edstate"] + 1e-30, "dstate")
    for key in ("y", "df", "dx"):
        assert (r[key][~r["used"]] == 7.0).all()


@pytest.mark.parametrize("n", [1, 64, 65, 1000, 262200])
def test_gated_scan_state_in_place(n):
    """The state written over the one taken in gives the bits of two buffers."""
    gen = _gen(22)
    ch = 136 if n < 2000 else 8
    gate, x, dy = (_normal(gen, torch.bfloat16, n, ch) for _ in range(3))
    cfg = raster.scan_config(torch.bfloat16, ch, True)
    docs = raster.documents(_ints([0]), _ints([n]), max_q_len=n)
    saved = _space(raster.gs_gated_scan_saved_size(cfg, docs, n))
    nf = raster.gs_gated_scan_fwd_workspace_size(cfg, docs, n)
    nb = raster.gs_gated_scan_bwd_workspace_size(cfg, docs, n)
    ws = _space(max(nf, nb))
    h0, dh = (torch.randn((1, ch), generator=gen, device="cuda") for _ in range(2))
    runs = []
    for same in (False, True):
        h, e = h0.clone(), dh.clone()
        ho, eo = (h, e) if same else (torch.empty_like(h), torch.empty_like(e))
        y, df, dx = (torch.empty_like(x) for _ in range(3))
        raster.gs_gated_scan_fwd(cfg, docs, n, gate, x, h, y, ho, saved, ws, nf)
        raster.gs_gated_scan_bwd(cfg, docs, n, gate, x, saved, dy, e, df, dx, eo, ws, nb)
        runs.append((y, ho, df, dx, eo))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_gated_scan_wrong_bound_is_only_slower():
    """max_q_len chooses the launch form; a document longer than it says is
    still computed."""
    gen = _gen(12)
    n, ch = 300, 16
    gate, x, dy = (_normal(gen, torch.float32, n, ch) for _ in range(3))
    cfg = raster.scan_config(torch.float32, ch, False)
    outs = []
    for bound in (0, 10):
        docs = raster.documents(_ints([0]), _ints([n]), max_q_len=bound)
        y, df, dx = (torch.empty_like(x) for _ in range(3))
        saved = _space(raster.gs_gated_scan_saved_size(cfg, docs, n))
        nb = raster.gs_gated_scan_bwd_workspace_size(cfg, docs, n)
        ws = _space(nb)
        raster.gs_gated_scan_fwd(cfg, docs, n, gate, x, None, y, None, saved, ws, nb)
        raster.gs_gated_scan_bwd(cfg, docs, n, gate, x, saved, dy, None, df, dx, None, ws, nb)
        outs.append((y, df, dx))
    ref = tu.scan_document(gate, x, torch.zeros(ch, device="cuda"), False, dy,
                           torch.zeros(ch, device="cuda"))
    for got in outs:
        for t, want, err in zip(got, (ref["y"], ref["df"], ref["dx"]),
                                (ref["ey"], ref["edf"], ref["edx"])):
            tu.close(t, want, err + 2.0 ** -24 * want.abs(), "bound")


@pytest.mark.parametrize("gate", [float("inf"), -float("inf"), 200.0, -200.0, 0.0])
def test_gated_scan_extreme_gates(gate):
    """An open gate keeps the state, a shut one takes the input."""
    n, ch = 70, 8
    f = torch.full((n, ch), gate, device="cuda")
    x = torch.randn((n, ch), generator=_gen(13), device="cuda")
    h0 = torch.full((1, ch), 3.0, device="cuda")
    cfg = raster.scan_config(torch.float32, ch, True)
    docs = raster.documents(_ints([0]), _ints([n]))
    y, end = torch.empty_like(x), torch.empty_like(h0)
    nb = raster.gs_gated_scan_fwd_workspace_size(cfg, docs, n)
    raster.gs_gated_scan_fwd(cfg, docs, n, f, x, h0, y, end, None, _space(nb), nb)
    if gate > 0:
        assert (y == 3.0).all() and (end == 3.0).all()
    elif gate < 0:
        assert torch.equal(y, x) and torch.equal(end[0], x[-1])
    else:
        ref = tu.scan_document(f, x, h0[0], True)
        tu.close(y, ref["y"], ref["ey"] + 2.0 ** -24, "y")


def test_gated_scan_repeats_bit_for_bit():
    a = _run_scan([1000, 16, 15], 256, True, torch.bfloat16)
    b = _run_scan([1000, 16, 15], 256, True, torch.bfloat16)
    for n in ("y", "df", "dx"):
        assert torch.equal(a[n][a["used"]], b[n][b["used"]])
    assert torch.equal(a["state"], b["state"]) and torch.equal(a["dstate"], b["dstate"])


def test_gated_scan_bad_channel_and_document_stay_alone():
    gen = _gen(14)
    lens, ch = [70, 80], 16
    starts, n = tu.starts_of(lens)
    gate, x = _normal(gen, torch.float32, n, ch), _normal(gen, torch.float32, n, ch)
    cfg = raster.scan_config(torch.float32, ch, True)
    docs = raster.documents(_ints(starts), _ints(lens))
    nb = raster.gs_gated_scan_fwd_workspace_size(cfg, docs, n)

    def run():
        y = torch.empty_like(x)
        raster.gs_gated_scan_fwd(cfg, docs, n, gate, x, None, y, None, None, _space(nb), nb)
        return y
    clean = run()
    x[3, 5] = float("nan")
    dirty = run()
    assert torch.isnan(dirty[3:70, 5]).all()
    dirty[3:70, 5] = clean[3:70, 5]
    assert torch.equal(clean, dirty)


def test_gated_scan_no_tokens():
    cfg = raster.scan_config(torch.float32, 8, True)
    h = torch.full((2, 8), 4.0, device="cuda")
    out = torch.zeros_like(h)
    docs = raster.documents(_ints([0, 0]), _ints([0, 0]))
    raster.gs_gated_scan_fwd(cfg, docs, 0, None, None, h, None, out, None, None, 0)
    assert torch.equal(h, out)
