"""Residual addition with root-mean-square norm and its adjoint, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring). The pages name no norm;
the reading is the usual pre-norm block: the stream h = x + res is stored, the
layer's input is y = h / sqrt(mean(h^2) + eps) * w. Pinned by a per-element
loop and by central finite differences.
"""
from __future__ import annotations

import numpy as np


def add_rmsnorm(x, res, w, eps: float, store):
    """(h, y, rs): h rounded by `store`, y and rs unrounded."""
    h = np.asarray(x, dtype=np.float64) if res is None else store(x + res)
    rs = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, h * rs[:, None] * w, rs


def add_rmsnorm_bwd(dy, h, w, rs, dh=None):
    """(dx, dw) for the stored h and the forward's rs."""
    n = h * rs[:, None]
    g = dy * w
    dx = rs[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return (dx if dh is None else dx + dh), np.sum(dy * n, axis=0)
