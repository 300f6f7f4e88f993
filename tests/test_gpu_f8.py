"""GPU parity of the e4m3 type: quantizer bytes and scales equal the oracle's, products within the bound
that the operations' roundings allow and within the normwise bound of the quantized kinds."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import f8
from tests.gpu_util import TOL_Q4_0, assert_close, say, to_dev, to_host

pytestmark = pytest.mark.gpu


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


def _bytes(t):
    import torch
    return to_host(t.view(torch.uint8))


def _act(rng, m, k):
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, rng.random(k) < 0.02] *= 20
    return x


def _weights(rng, n, k):
    return (rng.standard_normal((n, k)) * 0.02).astype(np.float32)


def bound(mag, k):
    """|error| of one output: a block's sum of at most 128 exact products, each addition off by at most one fp32
    step of the magnitudes' sum (2^-23, which also covers truncation), the scale product, the fma of each
    block, the join of at most 16 waves and 16 slices."""
    return (128 + 2 * (-(-k // 128)) + 32) * 2.0 ** -23 * mag


def check(y, w, ws, a, a_s, what):
    ref, mag = f8.mul_mat(w, ws, a, a_s)
    err = np.abs(y - ref)
    assert np.all(err <= bound(mag, w.shape[1])), f"{what}: {np.max(err / np.maximum(mag, 1e-300)):.3e} of the terms' sum"
    assert_close(y, ref, TOL_Q4_0, what)


@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 160), (5, 224), (37, 4128), (130, 128), (257, 288)])
@pytest.mark.parametrize("r", [1, 128])
def test_quantize_equals_oracle(rows, k, r):
    qs = _qs()
    say("quantize_f8", rows, k, r)
    x = _act(np.random.default_rng(rows * 1000 + k), rows, k)
    x[0, :min(k, 128)] = 0
    codes, scales = qs.quantize_f8(to_dev(x), r)
    wc, wsc = f8.quantize(x, r)
    assert np.array_equal(to_host(scales), wsc)
    assert np.array_equal(_bytes(codes), wc)


def test_quantize_edge_values():
    """Zero, subnormal, largest and non-finite blocks, every tie between two codes."""
    qs = _qs()
    say("quantize_f8 edges")
    x = np.zeros((8, 160), np.float32)
    x[1] = 2.0 ** -140
    x[2] = np.float32(3e38) * np.linspace(-1, 1, 160).astype(np.float32)
    x[3, 5] = np.inf
    x[3, 6] = 2
    x[4, 7] = np.nan
    x[4, 8] = -5
    x[5, :126] = f8._MID.astype(np.float32)[:126]         # 448 sets d = 1 below
    x[5, 126] = 448
    x[6] = -x[5]
    x[7] = np.float32(2.0 ** -126) * np.arange(160)
    codes, scales = qs.quantize_f8(to_dev(x), 1)
    wc, wsc = f8.quantize(x, 1)
    assert np.array_equal(to_host(scales), wsc)
    got = _bytes(codes)
    nan = wc & 0x7f == 0x7f
    assert np.array_equal(got & 0x7f == 0x7f, nan) and np.array_equal(got[~nan], wc[~nan])


# the fused kernel's rounds, the skinny kernel's row tiles, every output tile of the tiled kernel and both sides of
# its thresholds, ragged N, K ending inside a block, one block, one row
@pytest.mark.parametrize("m,n,k", [
    (1, 4096, 4096), (1, 1, 32), (1, 17, 96), (2, 300, 4128), (4, 129, 256), (5, 1000, 4128), (16, 257, 1024),
    (17, 130, 2080), (32, 64, 4096), (33, 48, 160), (64, 333, 1056), (65, 129, 128), (100, 515, 2080),
    (128, 256, 14336), (129, 257, 288), (300, 700, 1184), (512, 1024, 4096), (1, 40, 131072), (4, 40, 131072),
    (8, 300, 4096), (8, 300, 4128), (16, 65, 2048), (9, 8192, 4096), (70, 8200, 4128), (200, 130, 8224),
    (260, 16500, 2080), (24, 1100, 4096), (25, 1100, 4096), (300, 16500, 2080), (600, 4200, 1056), (1100, 4200, 160), (40, 33000, 160),
    (1, 16500, 160), (4, 8200, 1056), (16, 12300, 2048), (2, 16500, 2080),
])
def test_products(m, n, k):
    qs = _qs()
    say("f8", m, n, k)
    rng = np.random.default_rng(m * 1_000_003 + n * 17 + k)
    w, ws = f8.quantize(_weights(rng, n, k), 128)
    x = _act(rng, m, k)
    a, a_s = f8.quantize(x, 1)
    wd, wsd = to_dev(w), to_dev(ws)
    y = to_host(qs.mul_mat_f8_f32(wd, wsd, to_dev(x)))
    check(y, w, ws, a, a_s, f"f8_f32 {m}x{n}x{k}")
    y8 = to_host(qs.mul_mat_f8_f8(wd, wsd, to_dev(a), to_dev(a_s)))
    check(y8, w, ws, a, a_s, f"f8_f8 {m}x{n}x{k}")


@pytest.mark.parametrize("m", [1, 3, 16, 40, 130])
def test_rows_do_not_depend_on_their_batch_and_nan_stays_in_its_row(m):
    """A src1 row with a NaN, one with an infinity: their outputs are NaN, every other row's finite; weight rows
    past N and src1 rows past M are not read into results: dst behind the last row stays as it was."""
    import torch
    qs = _qs()
    say("f8 nan rows", m)
    rng = np.random.default_rng(m)
    n, k = 200, 416
    w, ws = f8.quantize(_weights(rng, n, k), 128)
    x = _act(rng, m, k)
    x[0, 3] = np.nan
    if m > 2:
        x[2, 400] = np.inf
    buf = torch.full((m + 2, n), 7.0, device="cuda")
    y = to_host(qs.mul_mat_f8_f32(to_dev(w), to_dev(ws), to_dev(x), out=buf[:m]))
    bad = [0, 2] if m > 2 else [0]
    good = [i for i in range(m) if i not in bad]
    assert np.isnan(y[bad]).all() and np.isfinite(y[good]).all()
    assert bool((buf[m:] == 7.0).all())
    if good:
        a, a_s = f8.quantize(x[good], 1)
        check(y[good], w, ws, a, a_s, f"good rows of {m}")


@pytest.mark.parametrize("m", [1, 16, 64, 130])
def test_nan_weight_reaches_its_column_only(m):
    qs = _qs()
    say("f8 nan weight", m)
    rng = np.random.default_rng(m + 50)
    n, k = 300, 288
    w, ws = f8.quantize(_weights(rng, n, k), 128)
    w[77, 280] = 0x7f
    w[150, 1] = 0xff
    y = to_host(qs.mul_mat_f8_f32(to_dev(w), to_dev(ws), to_dev(_act(rng, m, k))))
    cols = np.isnan(y).any(axis=0)
    assert np.isnan(y[:, [77, 150]]).all() and cols.sum() == 2


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (16, 1000, 4096), (64, 4096, 1024), (128, 4096, 14336)])
def test_graph_replays_and_a_second_stream_give_the_eager_bits(m, n, k):
    """Captured and replayed three times with eager work in between, and run on two streams with workspaces of
    their own: the same bits every time."""
    import torch
    qs = _qs()
    say("f8 graph", m, n, k)
    rng = np.random.default_rng(m + n)
    w, ws = (to_dev(v) for v in f8.quantize(_weights(rng, n, k), 128))
    x = to_dev(_act(rng, m, k))
    nbytes = max(qs.f8_workspace_size(m, n, k), 1)
    want = qs.mul_mat_f8_f32(w, ws, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, wsp = torch.empty_like(want), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qs.mul_mat_f8_f32(w, ws, x, out=out, ws=wsp)
    for rep in range(3):
        out.fill_(float("nan"))
        other = qs.mul_mat_f8_f32(w, ws, x * 2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
    assert torch.isfinite(other).all()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    torch.cuda.synchronize()
    for st in (s1, s2):
        with torch.cuda.stream(st):
            got.append([qs.mul_mat_f8_f32(w, ws, x) for _ in range(4)])
    torch.cuda.synchronize()
    for ys in got:
        for y in ys:
            assert torch.equal(y, want)


@pytest.mark.parametrize("m", [2, 20, 200])
def test_unaligned_dst_and_k_zero(m):
    import torch
    qs = _qs()
    say("f8 dst off 16", m)
    rng = np.random.default_rng(m)
    n, k = 264, 512
    w, ws = f8.quantize(_weights(rng, n, k), 128)
    x = _act(rng, m, k)
    a, a_s = f8.quantize(x, 1)
    buf = torch.full((m * n + 2,), 7.0, device="cuda")
    out = buf[1:-1].view(m, n)                                # 4-byte aligned only
    y = to_host(qs.mul_mat_f8_f32(to_dev(w), to_dev(ws), to_dev(x), out=out))
    check(y, w, ws, a, a_s, "dst off 16")
    assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0
    z = qs.mul_mat_f8_f32(torch.empty((n, 0), dtype=torch.uint8, device="cuda"), torch.empty((3, 0), device="cuda"),
                          torch.empty((m, 0), device="cuda"), out=out)
    assert not to_host(z).any()


def test_large_weights_past_4_gib():
    """Weight bytes past 2^32: sampled rows against the oracle."""
    import torch
    qs = _qs()
    n, k = 1_100_000, 4096
    say("f8 large", n, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = torch.randint(0, 0x7f, (n, k), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.rand((-(-n // 128), k // 128), device="cuda", generator=g) * 1e-3
    rows = np.r_[0:4, 524286:524290, 1048574:1048578, n - 4:n]
    for m in (1, 16, 70):
        x = torch.randn((m, k), device="cuda", generator=g)
        y = to_host(qs.mul_mat_f8_f32(w, ws, x)[:, rows])
        a, a_s = f8.quantize(to_host(x), 1)
        wv = np.stack([f8.VALUES[to_host(w[int(r)])] * np.repeat(to_host(ws[int(r) // 128]).astype(np.float64), 128) for r in rows])
        av = f8.dequantize(a, a_s, 1)
        err = np.abs(y - av @ wv.T)
        assert np.all(err <= bound(np.abs(av) @ np.abs(wv).T, k)), m


def test_both_stream_queries_name_the_current_stream():
    import torch
    qs = _qs()
    say("f8 streams")
    st = torch.cuda.Stream()
    assert qs._raw_stream(0) == qs._public_stream(0)
    with torch.cuda.stream(st):
        assert qs._raw_stream(0) == qs._public_stream(0) == st.cuda_stream


# What the shapes of test_products leave out, with the plan that each is here for (tests/test_f8_moe_host.py holds the
# plans to these, and the shapes of both lists to every kind of plan): (kernel, quantization rounds) or (tiled kernel's src1
# and weight rows, K slices, blocks of 128 per slice).
PLANNED = [
    ((1, 300, 7168), ("fused", 2)), ((2, 12400, 2592), ("fused", 2)), ((8, 12400, 2560), ("fused", 8)),
    ((24, 1030, 2080), ("skinny", 2)),
    ((25, 40, 8224), (64, 64, 13, 5)), ((3, 1100, 16384), (64, 64, 13, 10)),
    ((40, 33000, 1024), (64, 128, 1, 8)), ((9, 2049, 16384), (64, 128, 15, 9)), ((30, 4100, 8224), (64, 128, 7, 10)),
    ((129, 8200, 4096), (128, 128, 1, 32)), ((257, 16500, 2048), (128, 256, 1, 16)),
    ((129, 2049, 16384), (128, 128, 7, 19)), ((200, 4100, 8224), (128, 128, 3, 22)), ((200, 4100, 8416), (128, 128, 3, 22)),
    ((160, 4096, 8192), (128, 128, 4, 16)),
    ((257, 2049, 16384), (128, 256, 9, 15)), ((300, 4100, 8224), (128, 256, 5, 13)), ((270, 4160, 8096), (128, 256, 5, 13)),
    ((390, 4100, 8416), (128, 256, 3, 22)), ((512, 4096, 8192), (128, 256, 4, 16)),
]


def _codes(rng, n, k):
    """Weight codes of every magnitude and both signs, no NaN, with scales."""
    w = rng.integers(0, 0x7f, (n, k), dtype=np.uint8) | (rng.integers(0, 2, (n, k), dtype=np.uint8) << 7)
    return w, (1e-4 * rng.uniform(0.75, 1.25, (-(-n // 128), -(-k // 128)))).astype(np.float32)


@pytest.mark.parametrize("m,n,k", [shape for shape, _ in PLANNED])
def test_products_of_every_plan(m, n, k):
    """Several K slices on each tile (the last one shorter, K ending inside a block), calls on either side of the rules."""
    import torch
    qs = _qs()
    say("f8 planned", m, n, k)
    rng = np.random.default_rng(m * 1_000_003 + n * 17 + k)
    w, ws = _codes(rng, n, k)
    x = _act(rng, m, k)
    a, a_s = f8.quantize(x, 1)
    wd, wsd = to_dev(w), to_dev(ws)
    y = qs.mul_mat_f8_f32(wd, wsd, to_dev(x))
    check(to_host(y), w, ws, a, a_s, f"f8_f32 {m}x{n}x{k}")
    y8 = qs.mul_mat_f8_f8(wd, wsd, to_dev(a), to_dev(a_s))
    check(to_host(y8), w, ws, a, a_s, f"f8_f8 {m}x{n}x{k}")
    assert torch.equal(y8, qs.mul_mat_f8_f8(wd, wsd, to_dev(a), to_dev(a_s)))


@pytest.mark.parametrize("n,k", [(300, 4128), (1100, 2048), (4200, 8224), (8300, 1184)])
def test_rows_agree_between_batches(n, k):
    """A src1 row by itself and in larger batches: the same bits wherever the same kernel sums K in the same slices (each
    kernel's order of blocks depends on K alone), otherwise within the two sums' bounds; and by f32 or by codes."""
    import torch

    from tests import plans
    qs = _qs()
    say("f8 batches", n, k)
    rng = np.random.default_rng(n + k)
    w, ws = _codes(rng, n, k)
    x = _act(rng, 300, k)
    a, a_s = f8.quantize(x, 1)
    wd, wsd, xd, ad, asd = (to_dev(v) for v in (w, ws, x, a, a_s))
    first, seen = None, {}
    for m in (1, 2, 5, 8, 16, 17, 24, 33, 64, 65, 129, 300):
        for given in (False, True):
            y = qs.mul_mat_f8_f8(wd, wsd, ad[:m], asd[:m]) if given else qs.mul_mat_f8_f32(wd, wsd, xd[:m])
            p = plans.f8(m, n, k, given)
            other = seen.setdefault((p.kind, p.kchunk), y)
            rows = min(m, other.shape[0])
            assert torch.equal(y[:rows], other[:rows]), (m, given, p)
            if m > other.shape[0]:
                seen[p.kind, p.kchunk] = y
            first = y if first is None else first
            _, mag = f8.mul_mat(w, ws, a[:1], a_s[:1])
            assert np.all(np.abs(to_host(y[:1]).astype(np.float64) - to_host(first)) <= 2 * bound(mag, k)), (m, given)
    assert len(seen) > 1


@pytest.mark.parametrize("m", [1, 24, 70])
@pytest.mark.parametrize("exponent", [-110, -100, 100, 118])
def test_smallest_and_largest_scales(m, exponent):
    """Activations near both ends of fp32's range on each kernel.  The scales' product is rounded once, to 2^-24 of itself
    (in bound()) or to 2^-150 below the normal range, which each block's sum then multiplies."""
    qs = _qs()
    say("f8 scales", m, exponent)
    rng = np.random.default_rng(m)
    n, k = 300, 1056
    w, ws = _codes(rng, n, k)
    x = np.ldexp(rng.uniform(-1, 1, (m, k)), exponent).astype(np.float32)
    a, a_s = f8.quantize(x, 1)
    ref, mag = f8.mul_mat(w, ws, a, a_s)
    assert np.all(mag < 2.0 ** 127)
    sums = np.abs(f8.VALUES[a]) @ np.abs(f8.VALUES[w]).T
    tol = bound(mag, k) + 2.0 ** -150 * sums + (k // 128 + 40) * 2.0 ** -149
    for y in (qs.mul_mat_f8_f32(to_dev(w), to_dev(ws), to_dev(x)),
              qs.mul_mat_f8_f8(to_dev(w), to_dev(ws), to_dev(a), to_dev(a_s))):
        assert np.all(np.abs(to_host(y) - ref) <= tol)
