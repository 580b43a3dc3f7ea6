"""RMS norm with the residual addition, its backward, and 8-bit rows, in
numpy: fp64, with fp32 only where a rounding is part of the definition.

bf16 tensors come and go as uint16 bit patterns; bf16 and fp32 roundings are
to nearest, ties to even.
"""

import numpy as np

from .nf4 import bf16_bits_to_f64, f32_to_bf16_bits


def stream(x_bits, res_bits=None):
    """h = bf16(fl32(x + res)) as bits (x itself without a residual)."""
    if res_bits is None:
        return np.array(x_bits)
    s = bf16_bits_to_f64(x_bits).astype(np.float32) + bf16_bits_to_f64(res_bits).astype(np.float32)
    return f32_to_bf16_bits(s)


def forward(h_bits, w_bits, eps):
    """(y, rstd) in fp64 from the stored stream h [m, d]."""
    h = bf16_bits_to_f64(h_bits)
    w = bf16_bits_to_f64(w_bits)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + float(np.float32(eps)))
    return h * rstd[:, None] * w, rstd


def backward(dy, h, w, rstd, dh=None):
    """(dx, dw) in fp64 for fp64 arguments: dy, h, dh [m, d], w [d], rstd [m]."""
    d = h.shape[1]
    g = dy * w
    r = rstd[:, None]
    dx = r * (g - h * r * r * (g * h).sum(axis=1, keepdims=True) / d)
    if dh is not None:
        dx = dx + dh
    return dx, (dy * h * r).sum(axis=0)


def codes(t):
    """int8 codes of fp32 rows t [m, d] and their amax [m] (fp64):
    rint(fl32(127 t / amax)); 0 in rows of zeros and in rows that hold a
    non-finite value, whose amax is NaN."""
    t = np.asarray(t, dtype=np.float32).astype(np.float64)
    bad = ~np.isfinite(t).all(axis=1)
    amax = np.abs(np.where(bad[:, None], 0.0, t)).max(axis=1)
    div = np.where(amax > 0, amax, 1.0)[:, None]
    # the fp64 quotient rounds to the fp32 quotient (53 >= 2 * 24 + 2 bits)
    q = np.rint((127.0 * np.where(bad[:, None], 0.0, t) / div).astype(np.float32))
    return q.astype(np.int8), np.where(bad, np.nan, amax)


def forward_int8(h_bits, w_bits, eps):
    """(codes int8 [m, d], scale fp64 [m]) of the norm's output."""
    with np.errstate(invalid="ignore", over="ignore"):
        h = bf16_bits_to_f64(h_bits).astype(np.float32)
        w = bf16_bits_to_f64(w_bits).astype(np.float32)
        q, amax = codes(h * w)
        _, rstd = forward(h_bits, w_bits, eps)
        return q, np.where(np.isnan(amax), np.nan, amax * rstd / 127.0)


def quantize(x_bits):
    """(codes int8 [m, k], scale fp64 [m]) of bf16 rows."""
    q, amax = codes(bf16_bits_to_f64(x_bits).astype(np.float32))
    return q, amax / 127.0
