"""The linear in 8-bit integers, in numpy: exact int64 sums, fp64 scales."""

import numpy as np


def linear(x_codes, x_scale, w_codes, w_scale):
    """y [m, n] in fp64 for int8 codes [m, k], [n, k] and fp32 scales [m], [n]."""
    # sums of at most 2^31 are exact in fp64
    acc = x_codes.astype(np.float64) @ w_codes.astype(np.float64).T
    with np.errstate(invalid="ignore"):
        return acc * x_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)[None, :]
