"""Pins of the norm oracle: a per-element loop, and central differences."""
import math

import numpy as np

from oracle.norm import add_rmsnorm, add_rmsnorm_bwd

EXACT = lambda a: np.asarray(a, dtype=np.float64)


def test_forward_is_the_loop():
    g = np.random.default_rng(1)
    x, res, w = g.standard_normal((3, 5)), g.standard_normal((3, 5)), g.standard_normal(5)
    h, y, rs = add_rmsnorm(x, res, w, 1e-3, EXACT)
    for t in range(3):
        row = [x[t, i] + res[t, i] for i in range(5)]
        r = 1 / math.sqrt(sum(v * v for v in row) / 5 + 1e-3)
        assert abs(rs[t] - r) < 1e-14
        for i in range(5):
            assert h[t, i] == row[i] and abs(y[t, i] - row[i] * r * w[i]) < 1e-14
    h, y, _ = add_rmsnorm(np.zeros((1, 5)), None, w, 1e-3, EXACT)
    assert not h.any() and not y.any()


def test_backward_is_the_difference_quotient():
    g = np.random.default_rng(2)
    x, res, w = g.standard_normal((3, 6)), g.standard_normal((3, 6)), g.standard_normal(6)
    dy, dh = g.standard_normal((3, 6)), g.standard_normal((3, 6))

    def loss(x, w):
        h, y, _ = add_rmsnorm(x, res, w, 1e-3, EXACT)
        return float((dy * y).sum() + (dh * h).sum())

    h, _, rs = add_rmsnorm(x, res, w, 1e-3, EXACT)
    dx, dw = add_rmsnorm_bwd(dy, h, w, rs, dh)
    e = 1e-5     # truncation e^2 times third derivatives of order 10, rounding 2^-52 / e: 1e-8 covers both
    for i in np.ndindex(3, 6):
        p = np.zeros((3, 6))
        p[i] = e
        assert abs((loss(x + p, w) - loss(x - p, w)) / (2 * e) - dx[i]) < 1e-8
    for i in range(6):
        p = np.zeros(6)
        p[i] = e
        assert abs((loss(x, w + p) - loss(x, w - p)) / (2 * e) - dw[i]) < 1e-8
