"""Global gradient norm and clipping coefficient, in fp64."""

import numpy as np


def norm(grads):
    """sqrt of the sum of squares over all arrays."""
    return float(np.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads)))


def coef(total, max_norm):
    """min(1, max_norm / (total + 1e-6))."""
    return min(1.0, float(np.float32(max_norm)) / (total + float(np.float32(1e-6))))
