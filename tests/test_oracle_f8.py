"""The e4m3 codec and the mixture-of-experts oracle against facts that do not come from them."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import f8, moe


def test_values_of_known_bytes():
    # 0x38 = 1.0, 0x7e = 448, 0x01 = 2^-9 (smallest subnormal), 0x08 = 2^-6 (smallest normal)
    for b, v in ((0x00, 0.0), (0x38, 1.0), (0xb8, -1.0), (0x7e, 448.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9),
                 (0x08, 2.0 ** -6), (0x39, 1.125), (0x40, 2.0)):
        assert f8.VALUES[b] == v
    assert np.isnan(f8.VALUES[0x7f]) and np.isnan(f8.VALUES[0xff])


def test_encode_inverts_values_and_matches_torch():
    import torch
    codes = np.array([b for b in range(256) if b & 0x7f != 0x7f], np.uint8)
    assert np.array_equal(f8.encode(f8.VALUES[codes]), codes)
    rng = np.random.default_rng(5)
    v = np.concatenate([rng.standard_normal(4096) * s for s in (1e-4, 0.01, 1, 100)]).astype(np.float32)
    v = np.concatenate([np.clip(v, -448, 448), f8._MID.astype(np.float32), -f8._MID.astype(np.float32)])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.encode(v), want)


def test_ties_go_to_the_even_code():
    # between 1.0 (0x38) and 1.125 (0x39); between 1.125 and 1.25 (0x3a)
    assert f8.encode(np.float32(1.0625)) == 0x38
    assert f8.encode(np.float32(1.1875)) == 0x3a
    # below half of the smallest subnormal: zero; the tie itself: zero (even)
    assert f8.encode(np.float32(2.0 ** -10)) == 0


@pytest.mark.parametrize("rows,k,r", [(3, 160, 1), (130, 288, 128), (1, 32, 128)])
def test_quantize_round_trip(rows, k, r):
    rng = np.random.default_rng(rows + k)
    x = (rng.standard_normal((rows, k)) * 3).astype(np.float32)
    codes, scales = f8.quantize(x, r)
    assert scales.shape == (-(-rows // r), -(-k // 128))
    y = f8.dequantize(codes, scales, r)
    d = np.repeat(np.repeat(scales, r, 0)[:rows], 128, 1)[:, :k]
    # half a step: 2^-4 of the value, or half the subnormal spacing; the quotient's own fp32 roundings on top
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, d * 2.0 ** -10) * (1 + 2.0 ** -20))
    # the largest magnitude of a block becomes the code 448
    assert np.abs(f8.VALUES[codes]).max() == 448


def test_quantize_zero_tiny_and_non_finite_blocks():
    x = np.zeros((4, 128), np.float32)
    x[1, 5] = 2.0 ** -140
    x[2, 7] = np.inf
    x[2, 8] = 1.0
    x[3, 9] = np.nan
    x[3, 10] = 448.0
    codes, scales = f8.quantize(x, 1)
    assert not codes[0].any() and scales[0, 0] == np.float32(2.0 ** -126)
    assert scales[1, 0] == np.float32(2.0 ** -126) and codes[1, 5] == 0       # 2^-14 of a step
    assert np.isinf(scales[2, 0]) and codes[2, 7] == 0x7f and codes[2, 8] == 0
    assert codes[3, 9] == 0x7f and codes[3, 10] == 0x7e and scales[3, 0] == 1.0


def test_moe_selection_ties_and_weights():
    x = np.array([[1.0, 0.0]], np.float32)
    router = np.array([[1, 0], [2, 0], [1, 0], [2, 0]], np.float32)
    ids, w = moe.select(x, router, 3, True)
    assert ids.tolist() == [[1, 3, 0]]
    e = np.exp([0.0, 0.0, -1.0])
    assert np.allclose(w, e / e.sum(), rtol=1e-15)
    _, w = moe.select(x, router, 3, False)
    assert np.allclose(w, e / (2 + 2 * np.exp(-1.0)), rtol=1e-15)


def test_moe_layer_is_the_single_expert_mlp():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 8))
    g, u, d = (rng.standard_normal(s) for s in ((1, 6, 8), (1, 6, 8), (1, 8, 6)))
    y, ids, w, err = moe.layer(x, np.zeros((1, 8)), g, u, d, 1, True, 0.0, 0.0)
    a = x @ g[0].T
    want = (a / (1 + np.exp(-a)) * (x @ u[0].T)) @ d[0].T
    assert np.allclose(y, want, rtol=1e-13) and np.all(ids == 0) and np.all(w == 1)


def test_error_of_split_activations():
    """The two-part form in NumPy's binary16 keeps to the bound at every distance from the block's largest value,
    reaches it, and does not keep 22 bits far below it."""
    rng = np.random.default_rng(4)
    v = (rng.uniform(-1, 1, (4000, 32)) * 2.0 ** -rng.integers(0, 34, (4000, 32))).astype(np.float32)
    v[:, 0] = rng.uniform(0.5, 1, 4000).astype(np.float32)
    v[0, :2] = 1, 2.0 ** -27 + 2.0 ** -39 * 0.99              # the part below the first is lost whole
    v *= (2.0 ** rng.integers(-60, 60, (4000, 1))).astype(np.float32)
    top = np.abs(v).max(axis=1, keepdims=True)
    shift = 15 - np.frexp(top)[1]                             # largest magnitude in [2^14, 2^15)
    xs = np.ldexp(v, shift)
    hi = xs.astype(np.float16)
    lo = (xs - hi.astype(np.float32)).astype(np.float16)
    err = np.abs(np.ldexp(hi.astype(np.float64) + lo.astype(np.float64), -shift) - v)
    bound = moe.act_error(v)
    assert np.all(err <= bound) and err[0, 1] > 0.98 * bound[0, 1]
    assert np.any(err > 2.0 ** -13 * np.abs(v))
    near = np.abs(v) >= 2.0 ** -17 * top
    assert np.all(err[near] <= 2.0 ** -22 * np.abs(v)[near])
