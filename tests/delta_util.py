"""Attention gradients where delta = sum_j p_j dp_j is taken without the
roundings of the outputs (under a distance bias, and for tokens that see at
most 64 keys): a bound that leaves those roundings out, and inputs where they
would be most of the error."""
import torch

import token_util as tu


def dominated(gen, lengths, heads_q, heads_k, dim, dtype, device):
    """q, k, v, do of [rows, heads, dim]: each token's scores are led by one
    key of its document, more than the others together by the factor of a
    rounding, so that o is nearly that key's value (whose rounding o repeats)
    while the gradient of the scores comes from the rest."""
    rows = sum(lengths)
    r = lambda h: torch.randn((rows, h, dim), generator=gen, device=device)
    k, v, do = r(heads_k), r(heads_k), r(heads_q)
    q = torch.empty_like(do)
    at = 0
    for n in lengths:
        for i in range(n):
            # a key that a causal token sees too
            j = at + (i * 7) % (i + 1)
            # score lead |k| |q| / sqrt(dim): enough for weights of the others
            # near the type's rounding (2^-9, 2^-12)
            lead = 11.0 if dtype == torch.bfloat16 else 13.0
            x = k[j].repeat_interleave(heads_q // heads_k, 0)
            q[at + i] = x * (lead * dim ** 0.5 / (x * x).sum(-1, keepdim=True))
        at += n
    return [t.to(dtype) for t in (q, k, v, do)]


def bounds(r, q, k, v, do, scale, dtype):
    """Bounds of the errors of dq and dk of one head before the sum over shared
    heads and the last rounding: r as tu.attention_head returns it.

    ds is rounded to the type (u |ds|), all else is fp32 (EPS32 of the absolute
    terms; delta is a sum over the row, so its terms are the row's).  Where
    delta is corrected afterwards by e, at most what the roundings of o and of
    the weights make of do.o, ds was rounded before the correction and p t for
    it: 2 u p t |e|."""
    u, tiny = tu.U[dtype], tu.TINY[dtype]
    e = (do.abs() * u * (r["o"].abs() + r["ao"])).sum(1, keepdim=True) * 1.1
    row = (do.abs() * r["ao"]).sum(1, keepdim=True)
    pt = r["p"] * r["t"].abs()
    err = u * r["ds"].abs() + 2.0 * u * pt * e + tu.EPS32 * (r["size"] + pt * row) + tiny
    err = torch.where(r["p"] > 0, err, torch.zeros_like(err))
    return abs(scale) * err @ k.abs(), abs(scale) * err.T @ q.abs()


def as_rounded(q, k, v, do, scale, softcap, slope, seen, away, dtype, sign):
    """dq and dk of one head as the kernels round them, from the delta of the
    rounded outputs, with its correction (sign 1), without (0) or with the
    correction's sign wrong (-1); and with the correction but for the share
    that has already gone into dq ("half")."""
    to = lambda t: t.to(dtype).double()
    r = tu.attention_head(q, k, v, do, scale, softcap, slope, seen, away)
    o = to(to(r["p"]) @ v)
    dp = do @ v.T
    delta = (do * o).sum(1, keepdim=True)
    e = (r["p"] * (dp - delta)).sum(1, keepdim=True)
    both = 0.0 if sign == 0 else -1.0 if sign == -1 else 1.0
    in_dq = 0.0 if sign == "half" else both
    ds = to(r["p"] * (dp - delta) * r["t"])
    dq = scale * (ds @ k - in_dq * e * (to(r["p"] * r["t"]) @ k))
    dk = scale * to(r["p"] * (dp - delta - both * e) * r["t"]).T @ q
    return to(dq), to(dk), r
