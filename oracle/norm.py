"""Oracle: the root-mean-square norm with the residual's addition, and its gradients.

TEST INFRASTRUCTURE (see the package docstring).

y = h w / sqrt(mean(h^2) + eps) over a row.  All arithmetic is fp64 on decoded
values; h is the stored sum of x and the residual (rounded by the caller).
"""
from __future__ import annotations

import numpy as np

F64 = np.float64


def rms_norm(h, w, eps):
    """y and the row factors r [T]."""
    h = np.asarray(h, F64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * r[:, None] * np.asarray(w, F64), r


def rms_norm_backward(h, w, eps, dy, dh=None):
    """dx [T, H] and dw [H] of sum(dy * y) + sum(dh * h)."""
    h, w, dy = (np.asarray(v, F64) for v in (h, w, dy))
    _, r = rms_norm(h, w, eps)
    u = h * r[:, None]
    g = dy * w
    dx = r[:, None] * (g - u * (g * u).mean(axis=1, keepdims=True))
    return dx if dh is None else dx + np.asarray(dh, F64), (dy * u).sum(axis=0)
