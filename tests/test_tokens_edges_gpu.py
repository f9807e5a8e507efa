"""Edges of the token operators' arguments: what a call may leave out, and
values at the ends of their ranges.  Tolerances are token_util's bounds."""
import pytest
import torch

import token_util as tu
from differentiable_rasterization_amd import raster

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _space(nbytes):
    return torch.full((max(int(nbytes), 256),), 0xAB, dtype=torch.uint8, device="cuda")


def _check_qk(rows, hq, hk, dim, rotary, norm, eps, dtype, positions, freq):
    """Both directions of the norm and rotary position, against 64 bits."""
    gen = _gen(rows + dim + hq)
    q, k, dyq, dyk = (_normal(gen, dtype, rows, h, dim) for h in (hq, hk, hq, hk))
    wq, wk = (1 + 0.2 * torch.randn(dim, generator=gen, device="cuda") if norm else None
              for _ in "qk")
    cfg = raster.qk_config(dtype, hq, hk, dim, rotary, False, norm, eps, 1.0)
    oq, ok, dq, dk = (torch.full_like(t, 7.0) for t in (q, k, q, k))
    dwq, dwk = (torch.full((dim,), 7.0, device="cuda") for _ in "qk")
    raster.gs_qk_norm_rope_fwd(cfg, rows, positions, freq, wq, wk, q, k, oq, ok)
    n = raster.gs_qk_norm_rope_bwd_workspace_size(cfg, rows)
    raster.gs_qk_norm_rope_bwd(cfg, rows, positions, freq, wq, wk, q, k, dyq, dyk, dq, dk, dwq,
                               dwk, _space(n), n)
    at = positions if positions is not None else torch.zeros(rows, dtype=torch.int32,
                                                             device="cuda")
    turn = tu.turn_matrix(at, freq, dim, rotary, False, 1.0)
    u = tu.U[dtype]
    # the bounds of test_tokens_gpu.test_qk_norm_rope: 4e-6 for fp32 of a sum of
    # dim squares, a root, three products and the angle
    for x, w, y, dy, dx, dw in ((q, wq, oq, dyq, dq, dwq), (k, wk, ok, dyk, dk, dwk)):
        want, size = tu.qk_forward(x, w, turn, eps)
        tu.close(y, want, u * want.abs() + 4e-6 * size + tu.TINY[dtype], "y")
        gx, agx, gw, agw = tu.qk_backward(x, w, turn, eps, dy)
        tu.close(dx, gx, u * gx.abs() + 8e-6 * agx + tu.TINY[dtype], "dx")
        if norm:
            tu.close(dw, gw, 3e-5 * agw, "dw")
        else:
            assert (dw == 7.0).all()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,hq,hk,dim", [(1, 1, 1, 8), (5, 4, 2, 64), (300, 5, 3, 96),
                                            (1200, 6, 2, 128)])
def test_qk_nothing_turned_needs_no_positions(rows, hq, hk, dim, dtype, norm):
    _check_qk(rows, hq, hk, dim, 0, norm, 1e-6, dtype, None, None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,hq,hk,dim", [(1, 1, 1, 64), (7, 5, 2, 128), (300, 5, 2, 128),
                                            (33, 3, 1, 24), (64, 9, 3, 96)])
def test_qk_norm_without_epsilon(rows, hq, hk, dim, dtype):
    """Head counts that do not fill a wavefront: what its idle lanes do must
    not reach the weight gradients (1 / sqrt(0 + eps) has no value there)."""
    gen = _gen(rows)
    positions = torch.randint(0, 5000, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    freq = torch.rand(8, generator=gen, device="cuda")
    _check_qk(rows, hq, hk, dim, 16, True, 0.0, dtype, positions, freq)


def test_qk_more_rows_than_a_launch_has_workgroups():
    """2^26 and a few tokens, a wavefront each, are more than 2^32 work items.
    Nothing is normed or turned, so the outputs are the inputs."""
    rows = (1 << 26) + 9
    cfg = raster.qk_config(torch.bfloat16, 1, 1, 8, 0, norm=False)
    row = torch.arange(rows, dtype=torch.int32, device="cuda")
    q = (row % 251).to(torch.bfloat16)[:, None, None].expand(rows, 1, 8).contiguous()
    k = (row % 241).to(torch.bfloat16)[:, None, None].expand(rows, 1, 8).contiguous()
    oq, ok = torch.zeros_like(q), torch.zeros_like(k)
    raster.gs_qk_norm_rope_fwd(cfg, rows, None, None, None, None, q, k, oq, ok)
    assert torch.equal(oq, q) and torch.equal(ok, k)


def test_attention_more_documents_than_a_launch_has_workgroups():
    """2^21 one-token documents of eight key heads: 2^24 workgroups and 2^32
    work items.  Each sees one key, so its output is that key's value."""
    docs, heads = (1 << 21) + 3, 8
    q = torch.ones((docs, heads, 8), dtype=torch.bfloat16, device="cuda")
    v = (torch.arange(docs * heads, dtype=torch.int32, device="cuda") % 253).to(torch.bfloat16)
    v = v.view(docs, heads, 1).expand(docs, heads, 8).contiguous()
    start = torch.arange(docs, dtype=torch.int32, device="cuda")
    cfg = raster.attention_config(torch.bfloat16, heads, heads, 8, 1.0, True)
    d = raster.documents(start, torch.ones_like(start), max_q_len=1)
    o = torch.zeros_like(q)
    n = raster.gs_attention_fwd_workspace_size(cfg, d, docs, docs)
    raster.gs_attention_fwd(cfg, d, docs, docs, q, q, v, o, None, _space(n), n)
    assert torch.equal(o, v)


def test_gated_scan_more_states_than_a_launch_has_workgroups():
    """One document past what a single pass is made for and 32,768 empty ones,
    of 8,192 channels: 2^24 workgroups of 256 compose the chunks' states.
    Open gates and no input keep every state."""
    docs, ch, n = (1 << 15) + 1, 8192, 262145 + 64
    lens = torch.zeros(docs, dtype=torch.int32, device="cuda")
    lens[docs - 2] = n
    start = torch.zeros_like(lens)
    gate = torch.full((1, ch), float("inf"), dtype=torch.bfloat16, device="cuda").expand(n, ch)
    x = torch.zeros((1, ch), dtype=torch.bfloat16, device="cuda").expand(n, ch)
    h = (torch.arange(docs * ch, dtype=torch.int32, device="cuda") % 257).float().view(docs, ch)
    y = torch.zeros((n, ch), dtype=torch.bfloat16, device="cuda")
    end = torch.full_like(h, -1.0)
    cfg = raster.scan_config(torch.bfloat16, ch, False)
    d = raster.documents(start, lens)
    nb = raster.gs_gated_scan_fwd_workspace_size(cfg, d, n)
    raster.gs_gated_scan_fwd(cfg, d, n, gate, x, h, y, end, None, _space(nb), nb)
    assert torch.equal(end, h)
    for at in (0, 63, 64, n - 1):
        assert torch.equal(y[at], h[docs - 2].to(torch.bfloat16))
