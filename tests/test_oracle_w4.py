"""Pins of the MXFP4 oracle: the format's table, exhaustive nearest-element
search, and the serving form against the training layer's oracle."""
import numpy as np

import oracle.moe as om
from oracle.numerics import round_bf16
from oracle.w4 import E2M1, e2m1_decode, e2m1_encode, experts, w4_dequantize, w4_quantize


def test_element_table():
    # OCP MX v1.0, FP4 E2M1: sign, two exponent bits (bias 1), one fraction bit
    for c in range(16):
        s, e, m = -1.0 if c & 8 else 1.0, (c >> 1) & 3, c & 1
        assert e2m1_decode(c) == s * (m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + m / 2))


def test_encode_is_the_nearest_element():
    for v in np.concatenate([np.linspace(-7, 7, 2801), -np.linspace(-7, 7, 2801)]):
        c = int(e2m1_encode(v))
        got, best = abs(e2m1_decode(c) - np.clip(v, -6, 6)), np.abs(np.concatenate([E2M1, -E2M1]) - np.clip(v, -6, 6)).min()
        assert got <= best + 1e-15, v
    ties = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (6.5, 7), (-5.0, 14), (-0.25, 8)]
    for v, c in ties:
        assert int(e2m1_encode(v)) == c, v


def test_blocks():
    g = np.random.default_rng(1)
    w = g.standard_normal((2, 96, 3)) * np.exp2(g.integers(-30, 30, (2, 1, 3)))
    w[0, :32, 1] = 0
    q, s = w4_quantize(w)
    v = w4_dequantize(q, s)
    assert s[0, 0, 1] == 0 and not v[0, :32, 1].any()
    for m in range(2):
        for b in range(3):
            for n in range(3):
                blk = w[m, 32 * b:32 * b + 32, n]
                amax = np.abs(blk).max()
                if amax == 0:
                    continue
                unit = 2.0 ** (int(s[m, b, n]) - 127)
                assert 4 * unit <= amax < 8 * unit
                # at most half the widest step (2 units), plus saturation from 8 to 6
                assert np.all(np.abs(v[m, 32 * b:32 * b + 32, n] - blk) <= np.where(np.abs(blk) > 6 * unit, 2, 1) * unit)


def test_serving_form_is_the_layer():
    g = np.random.default_rng(2)
    T, d, E, k, F = 9, 12, 4, 2, 8
    x = round_bf16(g.standard_normal((T, d)))
    ws = [g.standard_normal(s) for s in ((E, d, F), (E, d, F), (E, F, d))]
    idx = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    p = g.random((T, k))
    exact = lambda a: np.asarray(a, dtype=np.float64)
    y, mag, _ = experts(x, idx, p, *ws, exact)
    fwd = om.layer_forward(dict(x=x, w_gate=ws[0], w_up=ws[1], w_down=ws[2], topk_idx=idx, topk_w=p), k, "f64")
    assert np.allclose(y, fwd["y"], rtol=1e-12, atol=1e-12) and np.all(np.abs(y) <= mag + 1e-12)
    idx[3] = -1
    idx[4, 0] = E
    add = g.standard_normal((T, d))
    y2, _, _ = experts(x, idx, p, *ws, exact, add)
    assert np.array_equal(y2[3], add[3]) and np.allclose(y2[5:], y[5:] + add[5:])
