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
