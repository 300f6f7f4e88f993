"""GPU parity of the experts for a given routing with 2 to 4 tokens, whose gate / up launch splits x in LDS: widths at which
the last round of its threads is partly filled, repeated experts, empty slots and NaN among several tokens."""
from __future__ import annotations

import numpy as np
import pytest

from tests import test_gpu_moe_routed as routed
from tests.gpu_util import say, to_dev, to_host

pytestmark = pytest.mark.gpu

KINDS = routed.KINDS

# tokens, D, F, experts, experts per token
HELD = [
    (4, 544, 64, 6, 3), (4, 640, 96, 16, 4), (4, 896, 64, 5, 5), (4, 1024, 64, 6, 2), (4, 1056, 64, 9, 2), (4, 1280, 160, 16, 16),
    (4, 1408, 64, 4, 1), (4, 1568, 64, 6, 3), (4, 1920, 64, 12, 3), (4, 1984, 64, 6, 3),
    (3, 672, 64, 6, 3), (3, 1280, 64, 5, 2), (3, 2048, 64, 5, 2), (3, 2688, 64, 4, 2),
    (2, 1056, 64, 6, 3), (2, 1920, 96, 5, 2), (2, 2048, 64, 5, 2), (2, 3968, 64, 4, 2),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,d,f,e,top_k", HELD)
def test_held(kind, t, d, f, e, top_k):
    qs = routed._qs()
    say("moe held", kind, t, d, f, e, top_k)
    m = routed.Layer(kind, d, f, e, top_k, t * 1000 + d + f)
    rng = np.random.default_rng(d + e)
    x, (ids, w) = routed._x(rng, t, d), routed._choice(rng, t, e, top_k)
    dst = m.check(x, ids, w, what=f"{kind} T={t} D={d} F={f} E={e} k={top_k}")
    again = qs.moe_routed_f32(m.layer, to_dev(x), to_dev(ids), to_dev(w))
    assert np.array_equal(to_host(again), dst)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,top_k", [(2, 3), (3, 8), (4, 5), (4, 9)])
def test_an_expert_named_several_times(kind, t, top_k):
    routed.test_an_expert_named_several_times(kind, t, top_k)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [2, 4])
def test_slots_without_an_expert(kind, t):
    routed.test_slots_without_an_expert(kind, t)


@pytest.mark.parametrize("kind", KINDS)
def test_nan_reaches_its_token_only(kind):
    """A NaN, an infinity and a NaN weight in one token of four each, in turn."""
    say("moe held nan", kind)
    qs = routed._qs()
    m = routed.Layer(kind, 640, 64, 5, 2, 3)
    rng = np.random.default_rng(1)
    x, (ids, w) = routed._x(rng, 4, 640), routed._choice(rng, 4, 5, 2)
    ref, err = m.oracle(x, ids, w)
    for bad in range(4):
        for what in range(3):
            xb, wb = x.copy(), w.copy()
            if what == 2:
                wb[bad, 1] = np.nan
            else:
                xb[bad, 639 if what else 130] = np.inf if what else np.nan
            dst = to_host(qs.moe_routed_f32(m.layer, to_dev(xb), to_dev(ids), to_dev(wb)))
            good = np.delete(np.arange(4), bad)
            assert np.isnan(dst[bad]).all(), (bad, what)
            assert np.all(np.abs(dst[good] - ref[good]) <= err[good]), (bad, what)


@pytest.mark.parametrize("kind", ["mxfp4", "f16"])
def test_graph_replays_follow_their_inputs(kind):
    routed.test_graph_replays_follow_their_inputs(kind, 4)


def test_two_streams_at_once():
    routed.test_two_streams_at_once(4)
