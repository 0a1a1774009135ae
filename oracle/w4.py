"""MXFP4 weights and the expert layer's serving form, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring). The format is the OCP
Microscaling v1.0 specification's: E2M1 elements (exponent bias 1, largest 6,
one subnormal 0.5, no infinities or NaN), one E8M0 scale per 32 values along
the contraction. Readings: X = floor(log2 amax) - 2 (2 is the exponent of 6),
at least -127 (also for an all-zero block); rounding to nearest, ties to even,
saturating at 6, the sign of a value that rounds to zero kept.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(v) -> np.ndarray:
    """Codes of float64 values: the nearest element, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), 6.0)
    hi = np.searchsorted(E2M1, a).clip(1, 7)           # E2M1[hi - 1] <= a <= E2M1[hi]
    lo = hi - 1
    d = (a - E2M1[lo]) - (E2M1[hi] - a)
    code = np.where(d > 0, hi, np.where(d < 0, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def e2m1_decode(codes) -> np.ndarray:
    c = np.asarray(codes).astype(np.int64)
    return np.where(c >> 3, -1.0, 1.0) * E2M1[c & 7]


def w4_quantize(w: np.ndarray):
    """(codes [M, K, N], scale codes [M, K/32, N]) of w [M, K, N], K % 32 == 0."""
    M, K, N = w.shape
    b = np.asarray(w, dtype=np.float64).reshape(M, K // 32, 32, N)
    amax = np.abs(b).max(axis=2)
    _, e = np.frexp(amax)
    x = np.where(amax > 0, np.maximum(e - 3, -127), -127)
    return e2m1_encode(np.ldexp(b, -x[:, :, None])).reshape(M, K, N), (x + 127).astype(np.uint8)


def w4_dequantize(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    M, K, N = codes.shape
    x = np.repeat(scales.astype(np.int64) - 127, 32, axis=1)
    return np.ldexp(e2m1_decode(codes), x)


def experts(x, topk_idx, topk_w, w_gate, w_up, w_down, store, y_add=None):
    """y of the serving form, expert by expert; also, for derived error bounds,
    sum_j |w| sum_f |H| |Wd| and the same with H's own error weights."""
    T, d = x.shape
    E, _, F = w_gate.shape
    y = np.zeros((T, d)) if y_add is None else np.array(y_add, dtype=np.float64)
    mag, hmag = np.zeros((T, d)), np.zeros((T, d))
    topk_idx = np.asarray(topk_idx)
    for e in range(E):
        t, j = np.nonzero(topk_idx == e)
        if not len(t):
            continue
        p, xe, ad = np.asarray(topk_w, dtype=np.float64)[t, j][:, None], x[t], np.abs(w_down[e])
        g, u = xe @ w_gate[e], xe @ w_up[e]
        s = 1 / (1 + np.exp(-g))
        h = store(g * s * u)
        np.add.at(y, t, p * (h @ w_down[e]))
        np.add.at(mag, t, np.abs(p) * (np.abs(h) @ ad))
        # |dH| per unit of relative error of the sums behind g and u (|silu'| < 1.1)
        ag, au = np.abs(xe) @ np.abs(w_gate[e]), np.abs(xe) @ np.abs(w_up[e])
        np.add.at(hmag, t, np.abs(p) * ((1.1 * ag * np.abs(u) + np.abs(g * s) * au) @ ad))
    return y, mag, hmag
