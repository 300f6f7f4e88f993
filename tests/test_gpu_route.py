"""GPU parity of the routing to experts: the oracle's experts, weights within a rounding to fp32 and fp64's own."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import route
from tests.gpu_util import say, to_dev, to_host

pytestmark = pytest.mark.gpu

# one rounding to fp32 (2^-24) and about a hundred of fp64
TOL = 2.0 ** -24 + 2.0 ** -44


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


def check(logits, top_k, bias=None, **kw):
    qs = _qs()
    r = qs.Router(logits.shape[1], top_k, bias=None if bias is None else to_dev(bias), **kw)
    ids, w = qs.route_f32(r, to_dev(logits))
    ri, rw = route.route(logits, top_k, bias=bias, **kw)
    ids, w = to_host(ids), to_host(w)
    nan = np.isnan(rw)
    assert np.array_equal(ids[~nan.any(axis=1)], ri[~nan.any(axis=1)])
    assert np.array_equal(np.isnan(w), nan)
    assert np.all(np.abs(w - rw)[~nan] <= TOL * np.abs(rw[~nan]) + 2.0 ** -149)
    return ids, w


@pytest.mark.parametrize("t,e,top_k", [(1, 1, 1), (1, 2, 2), (3, 5, 5), (1, 64, 8), (7, 65, 3), (130, 128, 6), (5, 129, 16),
                                       (9, 256, 8), (33, 300, 64), (4, 512, 64), (2, 511, 1), (1025, 60, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route(t, e, top_k, score, with_bias):
    say("route", t, e, top_k, score, with_bias)
    rng = np.random.default_rng(t * 7 + e + top_k)
    l = (3 * rng.standard_normal((t, e))).astype(np.float32)
    bias = (0.3 * rng.standard_normal(e)).astype(np.float32) if with_bias else None
    check(l, top_k, bias, score=score)
    check(l, top_k, bias, score=score, norm=False, scale=2.5)


@pytest.mark.parametrize("e,groups,group_k,group_top,top_k", [
    (256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (64, 64, 5, 2, 5), (64, 64, 5, 1, 5), (6, 3, 2, 2, 4), (100, 5, 1, 2, 20), (33, 11, 4, 2, 12),
    (512, 2, 1, 2, 16), (10, 10, 10, 1, 3), (49, 7, 2, 1, 14), (120, 40, 3, 2, 9)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(e, groups, group_k, group_top, top_k, score):
    say("route groups", e, groups, group_k, group_top)
    rng = np.random.default_rng(e + groups)
    l = (2 * rng.standard_normal((50, e))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(e)).astype(np.float32)
    ids, _ = check(l, top_k, bias, score=score, groups=groups, group_k=group_k, group_top=group_top)
    assert all(len(set(r[r >= 0] // (e // groups))) <= group_k for r in ids)


def test_ties_take_the_lower_index():
    say("route ties")
    rng = np.random.default_rng(0)
    l = rng.integers(0, 3, (64, 300)).astype(np.float32)
    check(l, 20)
    check(l, 20, score="sigmoid")
    check(l, 20, groups=30, group_k=4, group_top=2)
    check(np.zeros((3, 130), np.float32), 64)
    # differences in the last bits of a float64 score
    l = np.float32(1) + np.arange(100, dtype=np.float32)[None] * np.float32(2) ** -23
    check(np.concatenate([l, l[:, ::-1]]), 10, score="sigmoid")


def test_large_logits_of_both_signs():
    say("route large logits")
    rng = np.random.default_rng(4)
    l = np.float32(2) ** rng.integers(-30, 30, (20, 70)).astype(np.float32) * rng.choice([-1, 1], (20, 70)).astype(np.float32)
    # a softmax that leaves one expert, the others by index among scores of 0
    check(l, 5)
    check(l, 5, score="softmax", norm=False)
    check(-np.abs(l), 5, score="sigmoid")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts(score):
    """Minus infinity in logits and bias: never chosen; slots without an expert; tokens without any."""
    say("route masked", score)
    rng = np.random.default_rng(2)
    l = rng.standard_normal((9, 40)).astype(np.float32)
    l[1, 3:] = -np.inf
    l[2] = -np.inf
    l[3, ::2] = -np.inf
    l[4, 39:] = -np.inf
    bias = np.zeros(40, np.float32)
    bias[[0, 7]] = -np.inf
    bias[11] = 100
    for kw in ({}, {"groups": 8, "group_k": 2, "group_top": 2}, {"groups": 8, "group_k": 7, "group_top": 1}, {"norm": False}):
        ids, w = check(l, 6, score=score, **kw)
        assert (ids[2] == -1).all() and not w[2].any() and (ids[1, 3:] == -1).all()
        ids, _ = check(l, 6, bias, score=score, **kw)
        assert not np.isin(ids, [0, 7]).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinite_logits_stay_in_their_token(score):
    say("route nan", score)
    rng = np.random.default_rng(3)
    l = rng.standard_normal((7, 70)).astype(np.float32)
    l[1, 5], l[2], l[4, 66] = np.nan, np.nan, np.inf
    l[5, :30], l[5, 40] = -np.inf, np.nan
    ids, w = check(l, 4, score=score)
    assert ((ids >= 0) & (ids < 70)).all()
    assert np.isnan(w[[1, 2, 5]]).all() and np.isnan(w[4]).all() == (score == "softmax")
    check(l, 4, score=score, groups=7, group_k=3, group_top=2)


def test_outputs_end_where_they_should_and_graph_replays():
    import torch
    qs = _qs()
    say("route graph")
    l = to_dev(np.random.default_rng(5).standard_normal((37, 96)).astype(np.float32))
    r = qs.Router(96, 5, score="sigmoid", groups=6, group_k=2, group_top=2)
    wi, ww = qs.route_f32(r, l)
    ids = torch.full((37 * 5 + 8,), 77, dtype=torch.int32, device="cuda")
    w = torch.full((37 * 5 + 8,), 77.0, device="cuda")
    oi, ow = ids[:-8].view(37, 5), w[:-8].view(37, 5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.route_f32(r, l, ids=oi, weights=ow)
    for _ in range(3):
        oi.fill_(-5)
        ow.fill_(float("nan"))
        qs.route_f32(r, l * 2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oi, wi) and torch.equal(ow, ww)
    assert bool((ids[-8:] == 77).all()) and bool((w[-8:] == 77).all())


def test_a_bias_given_other_storage_is_read_there():
    import torch
    qs = _qs()
    say("route bias moved")
    l = torch.zeros((1, 10), device="cuda")
    b = torch.zeros(10, device="cuda")
    r = qs.Router(10, 1, bias=b)
    assert int(qs.route_f32(r, l)[0]) == 0
    b.data = torch.arange(10, device="cuda", dtype=torch.float32)
    assert int(qs.route_f32(r, l)[0]) == 9


def test_many_tokens():
    import torch
    qs = _qs()
    t, e = 1 << 22, 300                                       # logits past 2^32 bytes
    say("route many", t, e)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    l = torch.randn((t, e), device="cuda", generator=g)
    ids, w = qs.route_f32(qs.Router(e, 7), l)
    for at in (0, (1 << 32) // (4 * e) - 4, t - 8):
        ri, rw = route.route(to_host(l[at:at + 8]), 7)
        assert np.array_equal(to_host(ids[at:at + 8]), ri) and np.all(np.abs(to_host(w[at:at + 8]) - rw) <= TOL * rw)
