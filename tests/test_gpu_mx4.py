"""GPU parity of the MXFP4 type: quantizer bytes equal the oracle's, values are exact, products are exact where the sums fit
fp32 and within the bound of their roundings otherwise."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import mx4
from tests.gpu_util import TOL_Q4_0, assert_close, say, to_dev, to_host

pytestmark = pytest.mark.gpu


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


def _act(rng, m, k):
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[:, rng.random(k) < 0.02] *= 20
    return x


def _codes(rng, n, k, spread=2):
    """Random codes and scale bytes within 2^+-spread of 1; what lies in the padding is 255 (it is not to be read)."""
    s = np.full((n, mx4.padded(k)), 255, np.uint8)
    s[:, :k // 32] = rng.integers(127 - spread, 128 + spread, (n, k // 32))
    return rng.integers(0, 256, (n, k // 2), dtype=np.uint8), s


def bound(mag, k):
    """|error| of one output: per 128 k one instruction's sum and the addition to the accumulator, each off by at most a few
    fp32 steps of the magnitudes' sum (8 of 2^-23 allowed, for alignment and truncation), the join of 8 waves and 16 slices."""
    return (8 * (-(-k // 64)) + 32) * 2.0 ** -23 * mag


def check(y, w, ws, a, a_s, what, exact=False):
    ref, mag = mx4.mul_mat(w, ws, a, a_s)
    if exact:
        # every partial sum is a multiple of 2^-6 (codes 1/2 each, scales from 2^-2) below 2^18: exact in fp32
        assert mag.max() < 2.0 ** 18
        assert np.array_equal(y, ref), f"{what}: {np.abs(y - ref).max():.3g}"
        return
    assert np.all(np.abs(y - ref) <= bound(mag, 2 * w.shape[1])), what
    assert_close(y, ref, TOL_Q4_0, what)


@pytest.mark.parametrize("rows,k", [(1, 32), (1, 4096), (3, 160), (5, 224), (37, 4128), (130, 128), (257, 288), (70, 96)])
def test_quantize_equals_oracle(rows, k):
    import torch
    qs = _qs()
    say("quantize_mxfp4", rows, k)
    x = _act(np.random.default_rng(rows * 1000 + k), rows, k)
    x[0, :min(k, 64)] = 0
    x *= 2.0 ** np.random.default_rng(k).integers(-100, 100, (rows, 1)).astype(np.float32)
    codes = torch.full((rows * k // 2 + 16,), 0xaa, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * mx4.padded(k) + 16,), 0xaa, dtype=torch.uint8, device="cuda")
    out = codes[:-16].view(rows, k // 2), scales[:-16].view(rows, mx4.padded(k))
    qs.quantize_mxfp4(to_dev(x), out=out)
    wc, wsc = mx4.quantize(x)
    assert np.array_equal(to_host(out[0]), wc) and np.array_equal(to_host(out[1]), wsc)
    assert bool((codes[-16:] == 0xaa).all()) and bool((scales[-16:] == 0xaa).all())
    assert np.array_equal(to_host(qs.dequantize_mxfp4(*out)), mx4.dequantize(wc, wsc).astype(np.float32))


def test_quantize_edge_values():
    """Zeros of both signs, subnormals, the largest numbers, non-finite blocks, every tie between two codes at both ends of
    the scales."""
    qs = _qs()
    say("quantize_mxfp4 edges")
    x = np.zeros((12, 160), np.float32)
    x[0, 1::2] = -0.0
    x[1] = 2.0 ** -140
    x[2] = np.float32(3.4e38) * np.linspace(-1, 1, 160).astype(np.float32)
    x[3, 5], x[3, 6], x[3, 70] = np.inf, 2, 3
    x[4, 7], x[4, 8], x[4, 159] = np.nan, -5, -np.inf
    for row, e in ((5, 0), (6, -100), (7, 120), (8, -127), (9, -149 + 2)):
        unit = np.float32(2.0) ** e if e > -127 else np.ldexp(np.float32(1), e)
        near = np.concatenate([mx4.MID, -mx4.MID, np.nextafter(mx4.MID.astype(np.float32), np.float32(9)),
                               np.nextafter(mx4.MID.astype(np.float32), np.float32(0))])
        x[row, :28] = near.astype(np.float32) * unit
        x[row, 28], x[row, 29] = 4 * unit, 7.9 * unit
    x[10] = np.float32(2.0 ** -126) * np.arange(160, dtype=np.float32)
    x[11, :32] = np.finfo(np.float32).tiny
    codes, scales = qs.quantize_mxfp4(to_dev(x))
    wc, wsc = mx4.quantize(x)
    assert np.array_equal(to_host(scales), wsc)
    assert np.array_equal(to_host(codes), wc)
    got, want = to_host(qs.dequantize_mxfp4(codes, scales)), mx4.dequantize(wc, wsc)
    assert np.array_equal(got, want.astype(np.float32), equal_nan=True)


def test_dequantize_every_scale_and_code():
    qs = _qs()
    say("dequantize_mxfp4 all")
    codes = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1))
    scales = np.full((256, 4), 127, np.uint8)
    scales[:, 0] = np.arange(256)
    got = to_host(qs.dequantize_mxfp4(to_dev(codes), to_dev(scales)))
    with np.errstate(over="ignore"):
        want = mx4.dequantize(codes, scales).astype(np.float32)          # 2^127 * 6: infinite
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[:255]), np.signbit(want[:255]))


# the fused kernel's rounds, the skinny kernel's row tiles, every output tile of the tiled kernel and both sides of
# its thresholds, ragged N, K ending inside a group or a stage, one block, one row
SHAPES = [
    (1, 4096, 4096), (1, 1, 32), (1, 17, 96), (2, 300, 4128), (4, 129, 256), (5, 1000, 4128), (16, 257, 1024),
    (17, 130, 2080), (32, 64, 4096), (33, 48, 160), (64, 333, 1056), (65, 129, 128), (100, 515, 2080), (16, 4096, 64),
    (128, 256, 7168), (129, 257, 288), (300, 700, 1184), (512, 1024, 4096), (8, 300, 4096), (8, 300, 4128),
    (16, 65, 2048), (9, 8192, 4096), (70, 8200, 4128), (200, 130, 7136), (260, 16500, 2080), (24, 1100, 4096),
    (25, 1100, 4096), (300, 16500, 2080), (600, 4200, 1056), (1100, 4200, 160), (40, 33000, 160), (1, 16500, 160),
    (4, 8200, 1056), (16, 12300, 2048), (2, 16500, 2080), (512, 20000, 544), (257, 20000, 1024), (1, 3000, 7168),
    (31, 5000, 352), (48, 4096, 4096), (64, 14336, 1024), (128, 4096, 4096), (256, 4096, 2048), (40, 40, 7200),
    # several stages of the largest tiles, the last one ragged; K split evenly and unevenly
    (500, 14300, 1120), (1000, 14200, 800), (33, 70, 19936), (40, 30, 16384), (129, 300, 16416), (200, 300, 24608),
    (300, 1001, 28672), (300, 2048, 28928), (33, 300, 28704), (33, 4100, 2080), (20, 9001, 4128), (64, 8190, 2336), (128, 4000, 1888),
]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(m, n, k):
    qs = _qs()
    say("mxfp4", m, n, k)
    rng = np.random.default_rng(m * 1_000_003 + n * 17 + k)
    w, ws = _codes(rng, n, k, 1)
    a, a_s = _codes(rng, m, k, 1)
    wd, wsd = to_dev(w), to_dev(ws)
    y = qs.mul_mat_mxfp4_mxfp4(wd, wsd, to_dev(a), to_dev(a_s))
    check(to_host(y), w, ws, a, a_s, f"mxfp4 {m}x{n}x{k}", exact=True)
    x = _act(rng, m, k)
    a, a_s = mx4.quantize(x)
    check(to_host(qs.mul_mat_mxfp4_f32(wd, wsd, to_dev(x))), w, ws, a, a_s, f"f32 {m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1, 1000, 4096), (16, 300, 4128), (32, 200, 2048), (64, 260, 4096), (200, 300, 4128),
                                   (300, 520, 1024)])
@pytest.mark.parametrize("spread", [8, 20])
def test_products_of_scales_far_apart(m, n, k, spread):
    qs = _qs()
    say("mxfp4 spread", m, n, k, spread)
    rng = np.random.default_rng(m + n + k + spread)
    w, ws = _codes(rng, n, k, spread)
    a, a_s = _codes(rng, m, k, spread)
    ref, mag = mx4.mul_mat(w, ws, a, a_s)
    y = to_host(qs.mul_mat_mxfp4_mxfp4(to_dev(w), to_dev(ws), to_dev(a), to_dev(a_s)))
    assert np.all(np.abs(y - ref) <= bound(mag, k))
    assert np.linalg.norm(y - ref) <= 1e-6 * np.linalg.norm(ref)


@pytest.mark.parametrize("m", [1, 24, 70, 300])
@pytest.mark.parametrize("exponent", [-70, 50])
def test_smallest_and_largest_scales(m, exponent):
    """Both operands near an end of the scales: the products reach fp32's ends, the smallest fall below its normal range."""
    qs = _qs()
    say("mxfp4 scales", m, exponent)
    rng = np.random.default_rng(m)
    n, k = 300, 1056
    w, ws = _codes(rng, n, k)
    a, a_s = _codes(rng, m, k)
    ws[:, :k // 32] = np.clip(ws[:, :k // 32].astype(int) + exponent, 0, 254)
    a_s[:, :k // 32] = np.clip(a_s[:, :k // 32].astype(int) + exponent, 0, 254)
    ref, mag = mx4.mul_mat(w, ws, a, a_s)
    assert np.all(mag < 2.0 ** 127)
    y = to_host(qs.mul_mat_mxfp4_mxfp4(to_dev(w), to_dev(ws), to_dev(a), to_dev(a_s)))
    # below the normal range a sum may lose up to one smallest normal number per instruction
    tol = bound(mag, k) + (k // 64 + 40) * 2.0 ** -126
    assert np.all(np.abs(y - ref) <= tol)


@pytest.mark.parametrize("m", [1, 3, 16, 20, 40, 130, 300])
@pytest.mark.parametrize("n,k", [(200, 416), (270, 2080)])
def test_rows_do_not_depend_on_their_batch_and_nan_stays_in_its_row(m, n, k):
    """A src1 row with a NaN, one with an infinity: their outputs are NaN, every other row's exact; dst behind the last row
    stays as it was."""
    import torch
    qs = _qs()
    say("mxfp4 nan rows", m, n, k)
    rng = np.random.default_rng(m)
    w, ws = _codes(rng, n, k, 1)
    x = mx4.VALUES[rng.integers(0, 16, (m, k))].astype(np.float32)
    x[:, ::32] = 4
    x[0, 3] = np.nan
    if m > 2:
        x[2, 400] = np.inf
    buf = torch.full((m + 2, n), 7.0, device="cuda")
    y = to_host(qs.mul_mat_mxfp4_f32(to_dev(w), to_dev(ws), to_dev(x), out=buf[:m]))
    bad = [0, 2] if m > 2 else [0]
    good = [i for i in range(m) if i not in bad]
    assert np.isnan(y[bad]).all()
    assert bool((buf[m:] == 7.0).all())
    if good:
        a, a_s = mx4.quantize(x[good])
        check(y[good], w, ws, a, a_s, f"good rows of {m}", exact=True)


@pytest.mark.parametrize("m", [1, 16, 24, 64, 130, 300])
def test_nan_weight_block_reaches_its_column_only(m):
    qs = _qs()
    say("mxfp4 nan weight", m)
    rng = np.random.default_rng(m + 50)
    n, k = 300, 288
    w, ws = _codes(rng, n, k)
    ws[77, 8] = 255
    ws[150, 0] = 255
    y = to_host(qs.mul_mat_mxfp4_f32(to_dev(w), to_dev(ws), to_dev(_act(rng, m, k))))
    cols = np.isnan(y).any(axis=0)
    assert np.isnan(y[:, [77, 150]]).all() and cols.sum() == 2


@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (16, 1000, 4096), (30, 2000, 4096), (64, 4096, 1024), (128, 4096, 4096),
                                   (300, 1000, 1024)])
def test_graph_replays_and_a_second_stream_give_the_eager_bits(m, n, k):
    """Captured and replayed three times with eager work in between, and run on two streams with workspaces of
    their own: the same bits every time."""
    import torch
    qs = _qs()
    say("mxfp4 graph", m, n, k)
    rng = np.random.default_rng(m + n)
    w, ws = (to_dev(v) for v in _codes(rng, n, k, 12))
    x = to_dev(_act(rng, m, k))
    nbytes = max(qs.mxfp4_workspace_size(m, n, k), 1)
    want = qs.mul_mat_mxfp4_f32(w, ws, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, wsp = torch.empty_like(want), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qs.mul_mat_mxfp4_f32(w, ws, x, out=out, ws=wsp)
    for rep in range(3):
        out.fill_(float("nan"))
        other = qs.mul_mat_mxfp4_f32(w, ws, x * 2)
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
            got.append([qs.mul_mat_mxfp4_f32(w, ws, x) for _ in range(4)])
    torch.cuda.synchronize()
    for ys in got:
        for y in ys:
            assert torch.equal(y, want)


@pytest.mark.parametrize("m", [2, 20, 200, 300])
def test_unaligned_dst_and_k_zero(m):
    import torch
    qs = _qs()
    say("mxfp4 dst off 16", m)
    rng = np.random.default_rng(m)
    n, k = 263, 512
    w, ws = _codes(rng, n, k, 1)
    a, a_s = _codes(rng, m, k, 1)
    buf = torch.full((m * n + 2,), 7.0, device="cuda")
    out = buf[1:-1].view(m, n)                                # 4-byte aligned only
    y = to_host(qs.mul_mat_mxfp4_mxfp4(to_dev(w), to_dev(ws), to_dev(a), to_dev(a_s), out=out))
    check(y, w, ws, a, a_s, "dst off 16", exact=True)
    assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0
    z = qs.mul_mat_mxfp4_f32(torch.empty((n, 0), dtype=torch.uint8, device="cuda"),
                             torch.empty((n, 0), dtype=torch.uint8, device="cuda"), torch.empty((m, 0), device="cuda"), out=out)
    assert not to_host(z).any()


def test_torch_types_of_codes_and_scales():
    import torch
    qs = _qs()
    if not hasattr(torch, "float4_e2m1fn_x2"):
        pytest.skip("this torch has no such types")
    say("mxfp4 torch types")
    rng = np.random.default_rng(3)
    w, ws = (to_dev(v) for v in _codes(rng, 50, 128))
    a, a_s = (to_dev(v) for v in _codes(rng, 3, 128))
    want = qs.mul_mat_mxfp4_mxfp4(w, ws, a, a_s)
    c, e = torch.float4_e2m1fn_x2, torch.float8_e8m0fnu
    assert torch.equal(want, qs.mul_mat_mxfp4_mxfp4(w.view(c), ws.view(e), a.view(c), a_s.view(e)))


def _large(n, k, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(126, 129, (n, mx4.padded(k)), dtype=torch.uint8, device="cuda", generator=g)
    return w, s


def test_large_weights_past_4_gib():
    """Weight bytes past 2^32: sampled rows against the oracle."""
    qs = _qs()
    n, k = 2_200_000, 4096
    say("mxfp4 large", n, k)
    w, ws = _large(n, k, 1)
    rows = np.r_[0:4, 1048574:1048578, 2097150:2097154, n - 4:n]
    for m in (1, 20, 70, 300):
        a, a_s = _large(m, k, m)
        y = to_host(qs.mul_mat_mxfp4_mxfp4(w, ws, a, a_s)[:, rows])
        ref, mag = mx4.mul_mat(to_host(w[rows]), to_host(ws[rows]), to_host(a), to_host(a_s))
        assert mag.max() < 2.0 ** 18 and np.array_equal(y, ref), m
        x = qs.dequantize_mxfp4(a, a_s)
        assert np.array_equal(to_host(qs.mul_mat_mxfp4_f32(w, ws, x)[:, rows]),
                              mx4.mul_mat(to_host(w[rows]), to_host(ws[rows]), *mx4.quantize(to_host(x)))[0]), m


def test_quantizer_past_its_grid_and_4_gib():
    """More groups than the quantizer's grid holds, values past 2^32 bytes: rows around each border and at the ends."""
    import torch
    qs = _qs()
    rows, k = (1 << 24) + 40, 128
    say("quantize_mxfp4 large", rows, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn((rows, k), device="cuda", generator=g)
    codes, scales = qs.quantize_mxfp4(x)
    y = qs.dequantize_mxfp4(codes, scales)
    for at in (0, (1 << 23) - 8, (1 << 24) - 8, rows - 16):
        part = slice(at, at + 16)
        wc, wsc = mx4.quantize(to_host(x[part]))
        assert np.array_equal(to_host(codes[part]), wc) and np.array_equal(to_host(scales[part]), wsc), at
        assert np.array_equal(to_host(y[part]), mx4.dequantize(wc, wsc).astype(np.float32)), at


@pytest.mark.parametrize("m,n", [(1, 40), (20, 40), (70, 130), (257, 256)])
@pytest.mark.parametrize("k", [1 << 23, (1 << 23) - 32])
def test_product_at_the_largest_k(m, n, k):
    """K = 2^23 with codes of +-1/2 and one scale: sums of multiples of 1/4 up to 2^21, exact in fp32."""
    import torch
    qs = _qs()
    say("mxfp4 largest k", m, n, k)
    g = torch.Generator(device="cuda")
    g.manual_seed(m)

    def codes(rows):
        c = torch.randint(0, 4, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        c = 0x11 + (c & 1) * 8 + (c >> 1) * 128
        return c, torch.full((rows, mx4.padded(k)), 127, dtype=torch.uint8, device="cuda")

    w, ws = codes(n)
    a, a_s = codes(m)
    y = qs.mul_mat_mxfp4_mxfp4(w, ws, a, a_s)
    ref = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for k0 in range(0, k, 1 << 19):
        at = slice(k0 // 2, min(k0 + (1 << 19), k) // 2)
        sign = lambda c: torch.stack((1 - (c[:, at] >> 3 & 1).double() * 2, 1 - (c[:, at] >> 7).double() * 2), dim=2).flatten(1)
        ref += sign(a) @ sign(w).t() / 4
    assert bool((y == ref).all())


def test_product_of_more_src1_rows_than_a_grid_has_in_y():
    import torch
    qs = _qs()
    m, n, k = 70_001, 130, 160
    say("mxfp4 many rows", m, n, k)
    w, ws = _large(n, k, 3)
    a, a_s = _large(m, k, 4)
    y = qs.mul_mat_mxfp4_mxfp4(w, ws, a, a_s)
    ref = qs.dequantize_mxfp4(a, a_s).double() @ qs.dequantize_mxfp4(w, ws).double().t()
    assert bool((y == ref).all())
    assert bool((qs.mul_mat_mxfp4_f32(w, ws, torch.zeros((m, k), device="cuda")) == 0).all())


LARGE_SPLIT = (700, 3001, 32768)


def test_product_split_over_the_largest_tile():
    """Sums of multiples of 2^-4 below 2^20: exact in fp32, in whatever order they are joined."""
    qs = _qs()
    m, n, k = LARGE_SPLIT
    say("mxfp4 split of the largest tile", m, n, k)
    w, ws = _large(n, k, 5)
    a, a_s = _large(m, k, 6)
    y = qs.mul_mat_mxfp4_mxfp4(w, ws, a, a_s)
    x, v = qs.dequantize_mxfp4(a, a_s).double(), qs.dequantize_mxfp4(w, ws).double()
    assert float((x.abs() @ v.abs().t()).max()) < 2.0 ** 20
    assert bool((y == x @ v.t()).all())
