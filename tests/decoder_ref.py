"""Plain 64-bit forms of the operators of bsq_decoder.h, for their tests, on the CPU, and the
error bounds that the kernels' roundings add up to."""
import numpy as np

U = 2.0 ** -24                                   # half a step of fp32, relative
BF16 = 2.0 ** -8


# ------------------------------------------------------------------ norm and rotation


def norm_rope(x, weight, eps, positions, inv_freq, interleaved):
    """(out, bound) of one of q and k: x [rows, heads, D] float64.

    A head's squares are summed by 8 fused steps a lane and 5 sums over lanes, scaled, offset
    and put through a reciprocal root of one step (2 U): the factor is off by (13 + 2) U / 2 + 2 U,
    and two products follow: 12 U of y.  Cosine and sine in 32 bits: the reduced angle (at most
    0.8) and four or five roundings of numbers up to 1, 4 U; the angle itself, in 64 bits, by
    2^-51 of it.  Products and their sum: 2 U.  Then half a step of BF16."""
    rows, heads, D = x.shape
    y = x
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    n = len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq[None]
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    p = np.arange(n) * 2 if interleaved else np.arange(n)
    r = p + 1 if interleaved else p + n
    out, size = y.copy(), np.abs(y) * 12 * U
    out[..., p] = y[..., p] * cos - y[..., r] * sin
    out[..., r] = y[..., r] * cos + y[..., p] * sin
    both = (np.abs(y[..., p]) + np.abs(y[..., r])) * (18 * U + np.abs(angle)[:, None] * 2.0 ** -50)
    size[..., p] = size[..., r] = both
    return out, np.abs(out) * BF16 + size * (1 + BF16) + 2.0 ** -133
