"""Root-mean-square norm with the residual's addition, in NumPy: v = fl32(x + residual); rstd = fl32(1 / sqrt(mean(v^2) +
eps)) from float64; y = fl32(fl32(v * rstd) * weight)."""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight=None, eps=1e-5, residual=None):
    """(y float32, v float32, y in float64 without y's own roundings)."""
    with np.errstate(all="ignore"):
        v = x if residual is None else (x + residual).astype(np.float32)
        d = v.astype(np.float64)
        root = 1 / np.sqrt(np.mean(d * d, axis=1, keepdims=True) + np.float64(np.float32(eps)))
        w = np.ones(x.shape[1], np.float32) if weight is None else weight
        y = ((v * root.astype(np.float32)).astype(np.float32) * w).astype(np.float32)
        return y, v, d * root * w.astype(np.float64)
