"""The MXFP4, norm and routing oracles pinned to facts that do not come from themselves."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4, norm, route


def test_values_are_the_formats():
    # sign, exponent (bias 1), fraction; exponent 0 is subnormal
    for c in range(16):
        e, m = (c >> 1) & 3, c & 1
        v = Fraction(m, 2) if e == 0 else Fraction(2 + m, 2) * 2 ** (e - 1)
        assert Fraction(mx4.VALUES[c]) == (-v if c & 8 else v)


def test_ties_go_to_the_even_code():
    assert mx4.encode(mx4.MID).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert mx4.encode(np.nextafter(mx4.MID, 10)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert mx4.encode(np.nextafter(mx4.MID, 0)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert mx4.encode(np.array([7.99, -7.99, -0.0, -0.1])).tolist() == [7, 15, 8, 8]


@pytest.mark.parametrize("exponent", [-149, -140, -127, -126, -125, -1, 0, 1, 5, 126, 127])
def test_scale_is_the_largest_that_reaches_four(exponent):
    """amax / scale lies in [4, 8), or the scale is the smallest."""
    x = np.zeros((1, 32), np.float32)
    for lead in (1.0, 1.25, 1.99):
        x[0, 7] = -np.float32(np.ldexp(lead, exponent))
        _, s = mx4.quantize(x)
        q = Fraction(float(abs(x[0, 7]))) / Fraction(2) ** (int(s[0, 0]) - 127)
        assert 4 <= q < 8 or (s[0, 0] == 0 and q < 4)


def test_nearest_value_by_brute_force():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 64)).astype(np.float32)
    codes, scales = mx4.quantize(x)
    v = mx4.dequantize(codes, scales)
    for i in range(3):
        for j in range(64):
            unit = Fraction(2) ** (int(scales[i, j // 32]) - 127)
            off = min(abs(Fraction(float(x[i, j])) - Fraction(c) * unit) for c in mx4.VALUES)
            assert abs(Fraction(float(x[i, j])) - Fraction(v[i, j])) == off


def test_representable_values_come_back():
    rng = np.random.default_rng(1)
    e = rng.integers(-20, 20, (4, 3))
    v = mx4.VALUES[rng.integers(0, 16, (4, 96))]
    v[:, ::32] = 4                                           # every block's scale is 2^e
    v *= 2.0 ** e.repeat(32, axis=1)
    x = v.astype(np.float32)
    assert np.array_equal(mx4.dequantize(*mx4.quantize(x)), x)


def test_a_block_with_an_infinity_or_nan_is_nan_and_padding_is_127():
    x = np.ones((3, 96), np.float32)
    x[0, 40] = np.inf
    x[1, 70] = np.nan
    codes, s = mx4.quantize(x)
    assert s.shape == (3, 4) and (s[:, 3] == 127).all()
    assert np.isnan(mx4.dequantize(codes, s)).reshape(3, 3, 32).all(axis=2).tolist() == [[0, 1, 0], [0, 0, 1], [0, 0, 0]]


def test_norm_of_known_rows():
    x = np.array([[3, -4], [0, 0]], np.float32)
    y, v, _ = norm.rms_norm(x, eps=0.25)
    assert np.allclose(y[0], x[0] / np.sqrt(12.75)) and not y[1].any() and v is x
    _, v, _ = norm.rms_norm(x, residual=x)
    assert np.array_equal(v, 2 * x)


def test_routing_by_hand():
    l = np.log(np.array([[1, 2, 3, 4, 10, 1, 1, 2]], np.float64)).astype(np.float32)
    ids, w = route.route(l, 2)
    assert ids.tolist() == [[4, 3]] and np.allclose(w, [[10 / 14, 4 / 14]], rtol=1e-6)
    ids, w = route.route(l, 2, norm=False)
    assert np.allclose(w, [[10 / 24, 4 / 24]], rtol=1e-6)
    # groups of four: 3 + 4 < 10 + 2 by two, 4 < 10 by one; a bias turns the choice but not the weight
    assert route.route(l, 2, groups=2, group_top=2)[0].tolist() == [[4, 7]]
    bias = np.zeros(8, np.float32)
    bias[0] = 5
    ids, w = route.route(l, 2, bias=bias, groups=2, group_top=1, score="sigmoid", norm=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[1 / 2, 4 / 5]], rtol=1e-6)
    # ties to the lower index, masked experts never
    l = np.zeros((1, 5), np.float32)
    l[0, 0] = -np.inf
    ids, w = route.route(l, 5)
    assert ids.tolist() == [[1, 2, 3, 4, -1]] and np.allclose(w, [[0.25] * 4 + [0]])
