"""Which kernel, tile and split a call of the MXFP4 product takes, and which launches the experts for a given routing: every
one of them is among the shapes that run on a GPU, and the plans hold what the kernels assume."""
from __future__ import annotations

import itertools

from tests import mx4_plans
from tests.test_gpu_moe_routed import ROUTED, WITH_ROUTER
from tests.test_gpu_mx4 import LARGE_SPLIT, SHAPES
from tests.test_gpu_norm import SHAPES as NORMS

PRODUCTS = SHAPES + [LARGE_SPLIT]
TILES = [(32, 32), (32, 64), (64, 64), (64, 128), (128, 128), (256, 128), (256, 256)]


def _variant(p):
    if p.kind == "fused":
        return p.kind, p.nt
    if p.kind == "skinny":
        return p.kind, p.nt, p.waves if p.nt == 1 else 8
    return p.kind, p.bm, p.bn, p.split > 1


def test_every_variant_has_a_shape_on_the_gpu():
    seen = {_variant(mx4_plans.mx4(*s, given)) for s in PRODUCTS for given in (False, True)}
    want = {("fused", r) for r in (1, 2, 4, 8)} | {("skinny", 1, w) for w in (1, 2, 4, 8)} | {("skinny", 2, 8)}
    want |= {("wide", bm, bn, split) for bm, bn in TILES for split in (False, True)}
    assert want <= seen, want - seen


def test_splits_and_last_stages_have_shapes_on_the_gpu():
    """Splits that cut K unevenly, and stages that K ends in, of one half (128 k) or both, for each tile."""
    plans = [(s, mx4_plans.mx4(*s, True)) for s in PRODUCTS]
    wide = [(s, p, -(-s[2] // 256)) for s, p in plans if p.kind == "wide"]
    assert any(p.split > 1 and stages % p.kchunk for _, p, stages in wide)
    assert any(p.split > 1 and stages % p.kchunk == 0 for _, p, stages in wide)
    for tile in TILES:
        assert any((p.bm, p.bn) == tile and s[2] % 256 for s, p, _ in wide), tile


def test_plans_hold_what_the_kernels_assume():
    for m, n, k, given in itertools.product((1, 2, 15, 16, 17, 32, 33, 64, 65, 200, 600, 5000), (1, 31, 300, 2049, 4097, 9000, 140000),
                                            (32, 96, 128, 1056, 4096, 4128, 28704, 1 << 20, 1 << 23), (False, True)):
        p = mx4_plans.mx4(m, n, k, given)
        what = (m, n, k, given, p)
        groups, stages = -(-k // 128), -(-k // 256)
        assert p.kind in ("fused", "skinny", "wide"), what
        assert 0 <= p.ws_bytes, what
        if p.kind == "fused":
            assert not given and m <= 16 and 1 <= m * groups <= 32 * p.nt and p.ws_bytes == 0 and 1 <= p.grid_n <= -(-n // 16), what
        elif p.kind == "skinny":
            assert m <= 16 * p.nt and p.nt in (1, 2) and p.waves in (1, 2, 4, 8) and p.grid_n == -(-n // 16), what
        else:
            assert (p.bm, p.bn) in TILES, what
            # every workgroup has a stage, and together they have all
            assert (p.split - 1) * p.kchunk < stages <= p.split * p.kchunk and p.split <= 16, what
            assert p.split == 1 or p.ws_bytes >= 4 * p.split * m * n, what
        if not given and p.kind != "fused":
            assert p.ws_bytes >= m * (k // 2 + 4 * groups), what


def test_norm_shapes():
    """Waves of a row and rows of a workgroup: at most 16 waves; every number of pieces a lane holds (1, 2, 4, more) on the GPU."""
    held = set()
    for t, d in NORMS:
        waves, rows = mx4_plans.norm(t, d)
        assert waves in (1, 2, 4, 8, 16) and rows == max(1, 4 // waves)
        held.add(min(5, -(-(-(-d // 8)) // (64 * waves))))
    assert {1, 2, 5} <= held and held & {3, 4}, held


def test_routed_experts():
    """Few tokens on both sides of what the gate / up kernel holds of x; with MXFP4 experts down with one and two tiles, one and
    two units of weights at a time, whole and in slices."""
    held = {(t == 1, bool(mx4_plans.routed(6, t, d, f, e, k).held)) for t, d, f, e, k in ROUTED if t <= 4}
    assert held == set(itertools.product((False, True), repeat=2))
    for t, d, f, e, k in ROUTED + WITH_ROUTER:
        for mm_type in (1, 4, 5, 6):
            p = mx4_plans.routed(mm_type, t, d, f, e, k)
            assert bool(p.held) == (t <= 4 and t * 4 * -(-d // 128) <= 256)
    many = [(t, mx4_plans.routed(6, t, d, f, e, k)) for t, d, f, e, k in ROUTED + WITH_ROUTER if t > 4]
    assert {p.rt for _, p in many} == {1, 2}
    assert {t > 48 for t, p in many if p.rt == 2} == {False, True}
    assert any(p.slices > 1 for _, p in many) and any(p.slices == 1 for _, p in many)
