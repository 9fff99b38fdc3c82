"""Pins of the microscaled 4-bit oracle: hand-worked blocks, the rounding against an
exhaustive nearest-value search in rationals, the layout, the router's order."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4_oracle as mx


def test_hand_worked_blocks():
    x = np.zeros((1, 64))
    x[0, :8] = [4.0, 0.25, 0.26, -0.75, 5.0, -2.5, 3.5, 7.9]   # max 7.9: E = 0
    x[0, 32] = 1.0                                              # E = -2: 1 / 2^-2 = 4
    x[0, 33] = -0.125                                           # 0.5
    c, b = mx.quantise(x)
    assert list(b[0]) == [127, 125]
    # 0.25 is halfway between 0 and 0.5 (even: 0), 0.75 between 0.5 and 1 (even: 1),
    # 5 between 4 and 6 (even: 4), 2.5 between 2 and 3 (even: 2), 3.5 -> 4; 7.9 saturates
    assert list(mx.values(c, b, 64)[0, :8]) == [4, 0, 0.5, -1, 4, -2, 4, 6]
    assert list(mx.values(c, b, 64)[0, 32:34]) == [1.0, -0.125]


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -130, 2.0 ** 125, 1e-45])
def test_rounding_is_nearest_even_in_rationals(scale):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((4, 32)) * scale).astype(np.float32).astype(np.float64)
    x[1, :5] = np.array([1.25, 1.75, 2.5, 3.5, 5.0]) * scale
    c, b = mx.quantise(x)
    for r in range(4):
        a = max(abs(Fraction(float(v))) for v in x[r])
        E = -127
        while E < 125 and a >= Fraction(2) ** (E + 3):
            E += 1
        assert b[r, 0] == (E + 127 if a > 0 else 0)
        for k in range(32):
            v = abs(Fraction(float(x[r, k]))) / Fraction(2) ** E
            d = [abs(v - Fraction(float(g))) for g in mx.GRID]
            best = [i for i in range(8) if d[i] == min(d)]
            want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
            assert c[r, k] & 7 == want


def test_edges_of_the_scale():
    x = np.zeros((4, 32))
    x[1, 3] = np.inf
    x[2, 3] = np.nan
    x[3, 0] = float(np.finfo(np.float32).max)
    c, b = mx.quantise(x)
    assert list(b[:, 0]) == [0, 255, 255, 252]
    assert np.isnan(mx.values(c, b, 32)[1:3]).all() and mx.values(c, b, 32)[3, 0] == 6 * 2.0 ** 125


def test_layout_of_codes_and_scales():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((131, 200))
    c, b = mx.quantise(x)
    p, t = mx.pack(c, b)
    assert p.size == mx.code_bytes(131, 200) and t.size == mx.scale_bytes(131, 200) == 2 * 2 * 512
    assert p[130, 99] == c[130, 198] | c[130, 199] << 4
    # row 130 = row 2 of the second row of tiles; block 5 = block 1 of the second tile
    assert t[(1 * 2 + 1) * 512 + 2 * 16 + 0 * 4 + 1] == b[130, 5]
    assert t[(0 * 2 + 0) * 512 + (70 % 32) * 16 + (70 // 32) * 4 + 3] == b[70, 3]


def test_router_order_and_probabilities():
    x = np.array([[1.0, 0.0], [np.nan, 0.0]])
    r = np.array([[2.0, 0], [3.0, 0], [2.0, 0], [3.0, 0], [1.0, 0]])
    ids, p = mx.route(x, r, 3, True)
    assert list(ids[0]) == [1, 3, 0] and list(ids[1]) == [0, 1, 2]
    e = np.exp([0.0, 0.0, -1.0])
    assert np.allclose(p[0], e / e.sum(), rtol=1e-14)
    ids, p = mx.route(x, r, 3, False)
    full = np.exp(np.array([2, 3, 2, 3, 1.0]) - 3)
    assert np.allclose(p[0], full[[1, 3, 0]] / full.sum(), rtol=1e-14)
