"""Plain 64-bit forms of the operators of serving in 8 and 4 bits, with the
errors that the kernels' roundings leave (u: half a step of the output type,
relative to the value; E: half a step of fp32)."""
import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24
LEAST_SPAN = 2.0 ** -116


def row_codes(x):
    """(codes, scale) of rows [..., channels] in 64 bits; a row without a finite
    largest magnitude has codes 0 and scale NaN."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    none, wrong = top < LEAST_SPAN, ~torch.isfinite(top)
    zero = torch.zeros_like(x)
    # 127 x is exact, and so is a quotient between two codes: ties are ties
    codes = torch.where(none | wrong, zero, torch.round(127.0 * x / top)) + 0.0
    scale = torch.where(none, torch.zeros_like(top), top / 127.0)
    return codes, torch.where(wrong, torch.full_like(top, float("nan")), scale)[..., 0]


def linear(x, w, w_scale, bias):
    """y and the size that its fp32 errors are relative to."""
    codes, scale = row_codes(x)
    y = (codes @ w.double().T) * scale[:, None] * w_scale.double()
    size = y.abs()
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    return y, size


def linear_error(y, size, dtype):
    """Roundings to fp32: of the sum, of two scales' product (and of the row's
    scale), of the product with the sum, and of the sum with the bias."""
    least = {torch.float16: 2.0 ** -25}.get(dtype, 1e-37)
    return U[dtype] * (y.abs() + 5 * E * size) + 5 * E * size + least


# ---------------------------------------------------------------------------
# Caches
# ---------------------------------------------------------------------------
def head_codes(x, bits):
    """(codes, low, step) of heads [..., dim] in 64 bits."""
    x = x.double()
    low, high = x.amin(-1), x.amax(-1)
    levels = 2.0 ** bits - 1.0
    span = high - low
    wrong = ~(span < 2.0 ** 127) | torch.isnan(x).any(-1)
    none = ~wrong & (span < LEAST_SPAN)
    codes = torch.round((x - low[..., None]) * levels / span[..., None])
    codes = torch.where((wrong | none)[..., None], torch.zeros_like(codes), codes)
    nan = torch.full_like(low, float("nan"))
    step = torch.where(none, torch.zeros_like(span), span / levels)
    return codes, torch.where(wrong, nan, low), torch.where(wrong, nan, step)


def unpack(codes, bits):
    """Codes [..., dim] of bytes: in 4 bits, word by word, element 2i in bits 4i,
    element 2i + 1 in bits 16 + 4i."""
    if bits == 8:
        return codes.double()
    b = codes.unflatten(-1, (-1, 4)).long()
    word = b[..., 0] + (b[..., 1] << 8) + (b[..., 2] << 16) + (b[..., 3] << 24)
    e = [word >> (4 * (i // 2) + 16 * (i % 2)) & 15 for i in range(8)]
    return torch.stack(e, -1).flatten(-2).double()


def pack(u, bits):
    if bits == 8:
        return u.to(torch.uint8)
    e = u.long().unflatten(-1, (-1, 8))
    word = sum(e[..., i] << (4 * (i // 2) + 16 * (i % 2)) for i in range(8))
    return torch.stack([word >> 8 * i & 255 for i in range(4)], -1).flatten(-2).to(torch.uint8)


class Cache:
    """A cache on the GPU with room around its rows: codes, low and step."""

    def __init__(self, rows, heads, dim, bits, head_major=False, spare=0, ld=None):
        t, size = torch, dim * bits // 8
        if head_major:
            self.codes = t.randint(0, 256, (heads, rows, size + spare), dtype=t.uint8,
                                   device="cuda").transpose(0, 1)[:, :, :size]
        else:
            self.codes = t.randint(0, 256, (rows, heads, size + spare), dtype=t.uint8,
                                   device="cuda")[:, :, :size]
        ld = rows if ld is None else ld
        self.low = t.full((heads, ld), 3.0, device="cuda")[:, :rows]
        self.step = t.full((heads, ld), 0.5, device="cuda")[:, :rows]
        self.bits, self.dim = bits, dim

    def fill(self, x, first=0):
        """Values x [rows, heads, dim] from a row on."""
        u, low, step = head_codes(x, self.bits)
        n = x.shape[0]
        self.codes[first:first + n] = pack(u, self.bits)
        self.low[:, first:first + n] = low.T.float()
        self.step[:, first:first + n] = step.T.float()
        return self

    def view(self):
        from differentiable_rasterization_amd import raster
        return raster.codes(self.codes, self.low, self.step, self.bits)

    def parts(self, rows, head):
        """(codes, low, step) of rows of one head in 64 bits."""
        return (unpack(self.codes[rows, head], self.bits), self.low[head, rows].double(),
                self.step[head, rows].double())


def cached_head(q, key, value, scale, softcap, slope, seen, away, bits, dtype):
    """One head of one document's tokens over keys and values given as (codes,
    low, step): (o, error of o, lse, error of lse), everything in 64 bits.

    Scores: the product of dim codes, each fp32 step off by E of the sum of
    absolute terms, and three more operations.  Weights p: the score's error, an
    exponential (4 E).  Sums: fp32 over the keys, in four chains of 32-key steps.
    Weights times step: half a step of fp16, or of its smallest numbers, 2^-25,
    where a weight of at least 2^8 stands in the sum."""
    u, low, step = key
    k = low[:, None] + step[:, None] * u
    s = (q @ k.T) * scale
    dim, n = q.shape[1], k.shape[0]
    # the operands' offsets: up to the whole range of codes
    size = abs(scale) * (q.abs() @ (step[:, None] * 2.0 ** bits + 0 * u).T +
                         q.abs().sum(1, keepdim=True) * (low.abs() + 2.0 ** bits * step)[None, :])
    err = (dim + 8) * E * size
    if softcap:
        s = softcap * torch.tanh(s / softcap)
        err = err + (4e-7 * softcap if softcap <= 64 else 4e-7 * s.abs())
    s = s - slope * away
    err = err + 4 * E * (slope * away + s.abs())
    s = s.masked_fill(~seen, float("-inf"))
    lse = torch.logsumexp(s, -1) if n else torch.full((q.shape[0],), float("-inf"),
                                                      dtype=torch.float64, device=q.device)
    none = ~seen.any(1) if n else torch.ones(q.shape[0], dtype=torch.bool, device=q.device)
    p = torch.exp(s - torch.where(none, torch.zeros_like(lse), lse)[:, None])
    p = torch.where(seen, p, torch.zeros_like(p))
    vu, vlow, vstep = value
    mid = 128.0 if bits == 8 else 8.0
    part = torch.where(vstep.isnan(), torch.zeros_like(vstep), vstep)[:, None] * (vu - mid)
    mean = torch.where(vlow.isnan(), torch.zeros_like(vlow), vlow + mid * vstep)
    v = part + mean[:, None]
    o = p @ v
    err = torch.where(seen, err, torch.zeros_like(err))
    e_lse = (p * err).sum(1) + (n / 128 + 16) * E + 4 * E * lse.abs()
    top = vstep[~vstep.isnan()].max() if n else 0.0
    e_o = (p * (err + 16 * E)) @ v.abs() + (p * err).sum(1, keepdim=True) * o.abs() + \
        ((2.0 ** -11 + (n / 128 + 16) * E) * p) @ part.abs() + \
        (n / 128 + 16) * E * (p @ (mean.abs()[:, None] + part.abs())) + \
        2.0 ** -33 * top * seen.double().sum(1, keepdim=True) * 2.0 ** bits
    least = 2.0 ** -25 if dtype == torch.float16 else 1e-37
    return o, U[dtype] * (o.abs() + e_o) + e_o + least, lse, e_lse
