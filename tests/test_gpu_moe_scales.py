"""GPU parity of the experts at the largest scales of weights that cannot overflow on the way: a block's 32 products of
activations scaled to below 2^15 are at most 32 * 448 * 2^15 < 2^28.9 in e4m3, 32 * 6 * 2^15 < 2^22.6 in MXFP4; times a scale of
2^99, of 2^105, they stay below 2^128."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import f8, mx4
from tests.gpu_util import say, to_dev, to_host
from tests.test_gpu_moe_routed import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["mxfp4", "f8"])
@pytest.mark.parametrize("t", [1, 4, 20])
def test_largest_scales_of_down(kind, t):
    """Every weight of down the largest code at that scale, every h the same value just below a power of two."""
    say("moe largest scales", kind, t)
    d, f, e = 160, 96, 3
    m = Layer(kind, d, f, e, 2, 5)
    # gate and up: every row the first one's, so that all of h is one value
    for i in (0, 1):
        for a in (m.dev[i], m.scales[i]):
            v = to_host(a)
            v[:] = v[:, :1]
            a.copy_(to_dev(v))
    codes, scales = to_host(m.dev[2]), to_host(m.scales[2])
    codes[:] = 0x77 if kind == "mxfp4" else 0x7e
    scales[:] = 105 + 127 if kind == "mxfp4" else 2.0 ** 99
    m.dev[2].copy_(to_dev(codes))
    m.scales[2].copy_(to_dev(scales))
    for i in range(3):
        pairs = zip(to_host(m.dev[i]), to_host(m.scales[i]))
        m.values[i] = np.stack([mx4.dequantize(*p) if kind == "mxfp4" else f8.dequantize(*p, 128) for p in pairs])
    # h is about gate x times up x over 2: of x of 2^-50, scaled to a fraction of 1.98
    x = np.random.default_rng(t).standard_normal((t, d)) * 2.0 ** -50
    for i in range(t):
        h = abs((m.values[0][1, 0] @ x[i]) * (m.values[1][1, 0] @ x[i])) / 2
        x[i] *= np.sqrt(1.98 / (2 * np.frexp(h)[0]))
    ids, w = np.full((t, 2), -1, np.int32), np.ones((t, 2), np.float32)
    ids[:, 0] = 1
    dst = m.check(x.astype(np.float32), ids, w, kind)
    assert np.isfinite(dst).all() and np.all(dst != 0)
