"""GPU parity of the norm at the ends of fp32's range, where rstd itself leaves it, and of the routing with NaN and infinite
biases."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import norm, route
from tests.gpu_util import say, to_dev, to_host

pytestmark = pytest.mark.gpu


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


@pytest.mark.parametrize("t,d", [(7, 64), (7, 4096), (600, 512), (3, 65536)])
def test_rows_whose_rstd_is_not_a_normal_number(t, d):
    """Rows of one magnitude (sums of squares are exact): below 2^-128 with eps 0 rstd is infinite, past 2^126 it is subnormal,
    rounded to a multiple of 2^-149."""
    qs = _qs()
    say("rms_norm ends of the range", t, d)
    rng = np.random.default_rng(d)
    mags = np.array([2.0 ** -149, 2.0 ** -130, 2.0 ** -129, 2.0 ** -127, 1.5 * 2.0 ** 126, 1.25 * 2.0 ** 127, 3.0e38])
    x = (mags[np.arange(t) % len(mags)][:, None] * rng.choice([-1, 1], (t, d))).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    want = norm.rms_norm(x, w, 0.0)[0]
    assert np.isinf(want[:3]).all() and np.isfinite(want[3:7]).all()
    got = to_host(qs.rms_norm_f32(to_dev(x), to_dev(w), 0.0)[0])
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine])
    # 1 / sqrt in fp64 may be off by a step, which may move rstd by one of fp32 (2^-149 where it is subnormal, else 2^-23 of
    # it), and with it each of the two roundings that follow (2^-23 of the value)
    step = (2.0 ** -149 * np.abs(x.astype(np.float64) * w) + 3 * 2.0 ** -23 * np.abs(want.astype(np.float64)))[fine]
    assert np.all(np.abs(got[fine].astype(np.float64) - want[fine]) <= step)
    # with eps they are ordinary rows
    got = to_host(qs.rms_norm_f32(to_dev(x[:3]), to_dev(w), 1e-5)[0])
    assert np.isfinite(got).all() and np.abs(got).max() < 1e-35


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [{}, {"groups": 6, "group_k": 2, "group_top": 2}, {"groups": 6, "group_k": 3, "group_top": 1}])
def test_nan_and_infinite_biases(score, groups):
    """A NaN bias: chosen after all others; plus infinity: before all others; a logit of minus infinity masks either."""
    qs = _qs()
    say("route biases", score, groups)
    rng = np.random.default_rng(9)
    l = rng.standard_normal((11, 72)).astype(np.float32)
    l[3, 5] = l[4, 20] = l[5, 9] = -np.inf
    l[6] = -np.inf
    bias = (0.1 * rng.standard_normal(72)).astype(np.float32)
    bias[[5, 6, 71]] = np.nan
    bias[[20, 33]] = np.inf
    bias[40] = -np.inf
    for top_k in (1, 6, 30, 64):
        ids, w = qs.route_f32(qs.Router(72, top_k, score=score, bias=to_dev(bias), **groups), to_dev(l))
        ri, rw = route.route(l, top_k, score=score, bias=bias, **groups)
        assert np.array_equal(to_host(ids), ri), top_k
        assert np.all(np.abs(to_host(w) - rw) <= (2.0 ** -24 + 2.0 ** -44) * rw + 2.0 ** -149), top_k
        assert not np.isin(ri, [40]).any() and (ri[6] == -1).all()


def test_weights_of_a_token_with_a_nan_are_nan_in_its_empty_slots_too():
    qs = _qs()
    say("route nan, empty slots")
    l = np.full((2, 8), -np.inf, np.float32)
    l[:, 3], l[1, 5] = 1, np.nan
    ids, w = (to_host(v) for v in qs.route_f32(qs.Router(8, 4), to_dev(l)))
    assert ids.tolist() == [[3, -1, -1, -1], [3, 5, -1, -1]]
    assert w[0].tolist() == [1, 0, 0, 0] and np.isnan(w[1]).all()
