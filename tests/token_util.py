"""Plain 64-bit forms of the token operators (torch, any device), with the
error each kernel output may have, derived from the roundings the kernels make:

  u      unit roundoff of the output type (a value is rounded to it once);
  EPS32  fp32 arithmetic, taken as relative to the sum of absolute terms: the
         products of up to 128 elements, an exponential of a score up to some
         tens (its error is the score's), and short sums: 2e-5.
"""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
EPS32 = 2e-5
# smallest step of a type near zero (fp16 weights below 2^-14 lose bits)
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -24}
# where a type's values end: fp16 results are multiples of 2^-24, and products
# of fp32 numbers below 2^-126 are zero (the correctly rounded result of a
# number down there is this far off)
LEAST = {torch.float32: 1e-34, torch.bfloat16: 1e-34, torch.float16: 2.0 ** -25}


def close(got, want, tol, what):
    tol = tol + LEAST.get(got.dtype, 0.0)
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError("%s: %d of %d off, first at %d: %r, should be %r within %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]),
            float(want.flatten()[i]), float(tol.expand_as(want).flatten()[i])))


# ---------------------------------------------------------------------------
# Norm and rotary position
# ---------------------------------------------------------------------------
def turn_matrix(positions, inv_freq, dim, rotary, interleaved, amplitude):
    """The rows' linear maps [rows, dim, dim] of the rotation."""
    rows = positions.numel()
    m = torch.eye(dim, dtype=torch.float64, device=positions.device).repeat(rows, 1, 1)
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        t = positions.double() * inv_freq[i].double()
        m[:, a, a] = m[:, b, b] = amplitude * torch.cos(t)
        m[:, b, a] = amplitude * torch.sin(t)
        m[:, a, b] = -amplitude * torch.sin(t)
    return m


def qk_forward(x, w, turn, eps):
    """x [rows, heads, dim], w [dim] or None (no norm); (y, tolerance terms)."""
    x = x.double()
    n = x
    if w is not None:
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y = torch.einsum("rij,rhj->rhi", turn, n)
    return y, torch.einsum("rij,rhj->rhi", turn.abs(), n.abs())


def qk_backward(x, w, turn, eps, dy):
    """dx, dw and the absolute sums their errors are relative to."""
    x, dy = x.double(), dy.double()
    dn = torch.einsum("rji,rhj->rhi", turn, dy)
    an = torch.einsum("rji,rhj->rhi", turn.abs(), dy.abs())
    if w is None:
        return dn, an, None, None
    w = w.double()
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g, ag = dn * w, an * w.abs()
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    adx = r * (ag + x.abs() * r * r * (ag * x.abs()).mean(-1, keepdim=True))
    return dx, adx, (dn * x * r).sum((0, 1)), (an * x.abs() * r).sum((0, 1))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def seen_and_away(lq, lk, causal, prefix, device):
    i = torch.arange(lq, device=device)[:, None] + lk - lq
    j = torch.arange(lk, device=device)[None, :]
    seen = (j <= i) | (j < prefix) if causal else torch.ones((lq, lk), dtype=torch.bool,
                                                             device=device)
    return seen, (i - j).abs().double()


def attention_head(q, k, v, do, scale, softcap, slope, seen, away):
    """One head of one document in 64 bits; q [lq, d], k, v [lk, d], do [lq, d]
    or None.  Outputs with the terms of their errors."""
    s = (q @ k.T) * scale
    t = torch.ones_like(s)
    if softcap:
        th = torch.tanh(s / softcap)
        s, t = softcap * th, 1.0 - th * th
    s = (s - slope * away).masked_fill(~seen, float("-inf"))
    none = ~seen.any(1) if s.shape[1] else torch.ones(s.shape[0], dtype=torch.bool,
                                                      device=s.device)
    if s.shape[1]:
        top = s.amax(1, keepdim=True)
        e = torch.exp(s - torch.where(none[:, None], torch.zeros_like(top), top))
        e[none] = 0.0
        total = e.sum(1, keepdim=True)
        p = torch.where(none[:, None], torch.zeros_like(e), e / total.clamp(min=1e-300))
        lse = torch.where(none, torch.full_like(top[:, 0], float("-inf")),
                          top[:, 0] + torch.log(total[:, 0].clamp(min=1e-300)))
    else:
        p = s
        lse = torch.full((s.shape[0],), float("-inf"), dtype=torch.float64, device=s.device)
    out = {"p": p, "lse": lse, "o": p @ v, "ao": p @ v.abs(), "none": none}
    if do is None:
        return out
    dp = do @ v.T
    delta = (do * out["o"]).sum(1, keepdim=True)
    ds = p * (dp - delta) * t
    out.update(dq=scale * ds @ k, dk=scale * ds.T @ q, dv=p.T @ do)
    # absolute terms: ds itself, the delta from rounded outputs, fp32 noise
    size = p * (do.abs() @ v.abs().T + delta.abs())
    out.update(ds=ds, t=t, size=size)
    return out


def attention_error(r, q, k, v, do, scale, dtype):
    """Bounds of the errors of dq, dk, dv of one head (before the sum over
    shared heads and the final rounding)."""
    u, tiny = U[dtype], TINY[dtype]
    # o was rounded, and so were the weights that made it
    ddelta = (do.abs() * u * (r["o"].abs() + r["ao"])).sum(1, keepdim=True)
    e = u * r["ds"].abs() + r["p"] * r["t"].abs() * ddelta * 1.1 + EPS32 * r["size"] + tiny
    e = torch.where(r["p"] > 0, e, torch.zeros_like(e))
    ev = (u + EPS32) * r["p"] + torch.where(r["p"] > 0, torch.full_like(e, tiny),
                                            torch.zeros_like(e))
    return (abs(scale) * e @ k.abs(), abs(scale) * e.T @ q.abs(), ev.T @ do.abs())


# ---------------------------------------------------------------------------
# Gated scan
# ---------------------------------------------------------------------------
# a and 1 - a: an exponential, a reciprocal and two products of fp32
GATE = 1e-6


def scan_document(gate, x, h0, coupled, dy=None, dh=None):
    """One document [len, channels] in 64 bits, step by step, with bounds of
    the fp32 errors: each step adds GATE times its terms."""
    f, x = gate.double(), x.double()
    a, z = torch.sigmoid(f), torch.sigmoid(-f)
    n = f.shape[0]
    h = h0.double()
    eh = torch.zeros_like(h)
    y, ey, before, ebefore = [], [], [], []
    for t in range(n):
        u = z[t] * x[t] if coupled else x[t]
        before.append(h)
        ebefore.append(eh)
        eh = a[t] * eh + GATE * (a[t] * h.abs() + u.abs())
        h = a[t] * h + u
        y.append(h)
        ey.append(eh)
    out = {"y": torch.stack(y) if n else x, "ey": torch.stack(ey) if n else x, "state": h,
           "estate": eh}
    if dy is None:
        return out
    dy = dy.double()
    e = dh.double()
    ee = torch.zeros_like(e)
    df, dx, edf, edx = [None] * n, [None] * n, [None] * n, [None] * n
    for t in range(n - 1, -1, -1):
        g = dy[t] + e
        eg = ee + GATE * (dy[t].abs() + e.abs())
        d = before[t] - x[t] if coupled else before[t]
        ad = before[t].abs() + (x[t].abs() if coupled else 0.0)
        az = a[t] * z[t]
        dx[t] = g * z[t] if coupled else g
        edx[t] = (eg + GATE * g.abs()) * (z[t] if coupled else 1.0)
        df[t] = g * d * az
        edf[t] = (eg * d.abs() + g.abs() * (ebefore[t] + 2.0 * GATE * ad)) * az
        ee = a[t] * (eg + GATE * g.abs())
        e = a[t] * g
    out.update(df=torch.stack(df) if n else x, dx=torch.stack(dx) if n else x,
               edf=torch.stack(edf) if n else x, edx=torch.stack(edx) if n else x, dstate=e,
               edstate=ee)
    return out


def starts_of(lengths, gap=0):
    out, at = [], 0
    for n in lengths:
        out.append(at)
        at += n + gap
    return out, max(at - gap, 0) if lengths else 0


def sqrt_scale(dim):
    return 1.0 / math.sqrt(dim)
