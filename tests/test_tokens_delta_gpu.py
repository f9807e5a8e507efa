"""The gradients of attention where delta is taken without the roundings of the
outputs, held to a bound that leaves those roundings out (delta_util; that the
bound fails without the correction is shown on the CPU in test_tokens_delta)."""
import pytest
import torch

import delta_util as du
import token_util as tu
from differentiable_rasterization_amd import raster

pytestmark = pytest.mark.gpu

CASES = [
    # lengths, heads_q, heads_k, dim, largest slope, softcap, causal
    ([60, 33, 58], 4, 2, 64, 0.01, 0.0, True),       # few columns: corrected at the end
    ([60, 33, 58], 4, 2, 128, 0.01, 30.0, False),
    ([120, 150], 2, 1, 96, 0.005, 0.0, True),
    ([60, 33, 58], 160, 80, 64, 0.01, 0.0, True),    # 128 columns, heads of 64: the same
    ([60, 33, 58], 160, 80, 40, 0.01, 30.0, False),
    ([150, 129, 31], 160, 160, 64, 0.004, 0.0, True),
    ([60, 33, 58], 160, 80, 128, 0.01, 0.0, True),   # 128 columns: a walk of its own
    ([150, 129, 31], 160, 80, 96, 0.004, 30.0, True),
    ([150, 129, 31], 160, 160, 128, 0.004, 0.0, False),
    ([60, 33, 64], 4, 2, 64, 0.0, 0.0, True),        # at most 64 keys: the same, short
    ([60, 33, 64], 4, 2, 128, 0.0, 0.0, False),
    ([64, 50, 64], 128, 64, 64, 0.0, 0.0, True),
    ([64, 50, 64], 128, 64, 128, 0.0, 0.0, False),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_gradients_without_the_outputs_roundings(case, dtype):
    lens, hq, hk, dim, steep, softcap, causal = case
    gen = torch.Generator(device="cuda").manual_seed(dim + hq)
    q, k, v, do = du.dominated(gen, lens, hq, hk, dim, dtype, "cuda")
    n, g, scale = len(q), hq // hk, tu.sqrt_scale(dim)
    slopes = torch.linspace(0.5 * steep, steep, hq, device="cuda") if steep else None
    cfg = raster.attention_config(dtype, hq, hk, dim, scale, causal, softcap, slopes)
    starts, _ = tu.starts_of(lens)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    docs = raster.documents(ints(starts), ints(lens))
    o, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
    lse = torch.zeros((hq, n), device="cuda")
    size = max(raster.gs_attention_fwd_workspace_size(cfg, docs, n, n),
               raster.gs_attention_bwd_workspace_size(cfg, docs, n, n), 256)
    ws = torch.empty((size,), dtype=torch.uint8, device="cuda")
    raster.gs_attention_fwd(cfg, docs, n, n, q, k, v, o, lse, ws, size)
    raster.gs_attention_bwd(cfg, docs, n, n, q, k, v, o, lse, do, dq, dk, dv, ws, size)
    wq, wk, eq, ek = (torch.zeros(t.shape, dtype=torch.float64, device="cuda")
                      for t in (q, k, q, k))
    for a, m in zip(starts, lens):
        at = slice(a, a + m)
        seen, away = tu.seen_and_away(m, m, causal, 0, "cuda")
        for h in range(hq):
            x, y, z, w = (t.double() for t in (q[at, h], k[at, h // g], v[at, h // g],
                                               do[at, h]))
            r = tu.attention_head(x, y, z, w, scale, softcap,
                                  float(slopes[h]) if steep else 0.0, seen, away)
            wq[at, h] = r["dq"]
            wk[at, h // g] += r["dk"]
            bq, bk = du.bounds(r, x, y, z, w, scale, dtype)
            eq[at, h] = bq
            ek[at, h // g] += bk
    tu.close(dq, wq, eq + tu.U[dtype] * wq.abs(), "dq")
    tu.close(dk, wk, ek + tu.U[dtype] * wk.abs(), "dk")
