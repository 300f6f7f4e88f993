"""GPU parity of the RMS norm: v equals the oracle's, y within the roundings of its three steps, codes and scales those of the
quantizers on the same y."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import norm
from tests.gpu_util import say, to_dev, to_host

pytestmark = pytest.mark.gpu

# rstd, v * rstd and the product with weight are each off by at most half a step (2^-24)
TOL = 3.01 * 2.0 ** -24


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


def _inputs(t, d, seed=0):
    rng = np.random.default_rng(seed + t * 131 + d)
    x = rng.standard_normal((t, d)).astype(np.float32) * np.float32(2) ** rng.integers(-8, 8, (t, 1)).astype(np.float32)
    r = (3 * rng.standard_normal((t, d))).astype(np.float32)
    w = (1 + 0.3 * rng.standard_normal(d)).astype(np.float32)
    return x, r, w


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 33), (4, 64), (7, 511), (9, 513), (2, 1000), (17, 2049), (1, 8192), (6, 16391),
          (3, 70001), (1, 262144), (600, 512), (513, 100), (700, 2056), (515, 5000), (520, 12288), (514, 40000), (4095, 128),
          (600, 1000), (2, 12000)]


@pytest.mark.parametrize("t,d", SHAPES)
def test_norm(t, d):
    import torch
    qs = _qs()
    say("rms_norm", t, d)
    x, r, w = _inputs(t, d)
    buf = torch.full((2, t * d + 8), 7.0, device="cuda")
    out, sum_out = buf[0, :-8].view(t, d), buf[1, :-8].view(t, d)
    qs.rms_norm_f32(to_dev(x), to_dev(w), 1e-5, residual=to_dev(r), out=out, sum_out=sum_out)
    _, v, exact = norm.rms_norm(x, w, 1e-5, r)
    assert np.array_equal(to_host(sum_out), v)
    assert np.all(np.abs(to_host(out) - exact) <= TOL * np.abs(exact) + 2.0 ** -149)
    assert bool((buf[:, -8:] == 7.0).all())


@pytest.mark.parametrize("t,d", [(2, 100), (600, 4096), (3, 40000)])
def test_arguments_that_may_be_left_out_and_sums_in_place(t, d):
    qs = _qs()
    say("rms_norm forms", t, d)
    x, r, w = _inputs(t, d, 5)
    near = lambda y, e: np.all(np.abs(to_host(y) - e) <= TOL * np.abs(e))
    y, v = qs.rms_norm_f32(to_dev(x))
    assert v is None and near(y, norm.rms_norm(x)[2])
    y, v = qs.rms_norm_f32(to_dev(x), to_dev(w), 0.5)
    assert v is None and near(y, norm.rms_norm(x, w, 0.5)[2])
    _, s, exact = norm.rms_norm(x, w, 1e-5, r)
    xd, rd = to_dev(x), to_dev(r)
    y, v = qs.rms_norm_f32(xd, to_dev(w), 1e-5, residual=rd, sum_out=rd)
    assert v is rd and np.array_equal(to_host(rd), s) and near(y, exact) and np.array_equal(to_host(xd), x)
    xd, rd = to_dev(x), to_dev(r)
    y, v = qs.rms_norm_f32(xd, to_dev(w), 1e-5, residual=rd, sum_out=xd)
    assert v is xd and np.array_equal(to_host(xd), s) and near(y, exact) and np.array_equal(to_host(rd), r)
    xd = to_dev(x)
    y, v = qs.rms_norm_f32(xd, sum_out=xd)                    # no residual: v = x
    assert np.array_equal(to_host(xd), x) and near(y, norm.rms_norm(x)[2])


@pytest.mark.parametrize("t,d", [(1, 32), (1, 4096), (3, 160), (5, 4128), (600, 512), (513, 2080), (515, 8192), (520, 16416),
                                 (2, 40032), (600, 96)])
def test_quantized_outputs_are_the_quantizers(t, d):
    """The same bytes as the norm in f32 followed by the quantizer, whatever lies behind the outputs untouched."""
    import torch
    qs = _qs()
    say("rms_norm quantized", t, d)
    x, r, w = (to_dev(v) for v in _inputs(t, d, 9))
    y, v = qs.rms_norm_f32(x, w, 1e-6, residual=r)
    ng = -(-d // 128)
    for kind, quantize, cols, sdtype, scols in ((qs.MM_TYPE_F8, qs.quantize_f8, d, torch.float32, ng),
                                                (qs.MM_TYPE_MXFP4, qs.quantize_mxfp4, d // 2, torch.uint8, 4 * ng)):
        codes = torch.full((t * cols + 16,), 0xaa, dtype=torch.uint8, device="cuda")
        scales = torch.full((t * scols + 4,), 77, dtype=sdtype, device="cuda")
        out = codes[:-16].view(t, cols), scales[:-4].view(t, scols)
        (c, s), v2 = qs.rms_norm_f32(x, w, 1e-6, residual=r, out_type=kind, out=out)
        wc, wsc = quantize(y)
        assert torch.equal(c, wc.view(torch.uint8)) and torch.equal(s, wsc) and torch.equal(v, v2)
        assert bool((codes[-16:] == 0xaa).all()) and bool((scales[-4:] == 77).all())


@pytest.mark.parametrize("d", [96, 4096, 40000])
def test_rows_with_infinities_and_nan_and_zeros(d):
    qs = _qs()
    say("rms_norm non-finite", d)
    x, _, w = _inputs(6, d, 3)
    x[1, 5], x[2, 6], x[3] = np.inf, np.nan, 0
    x[4] = np.float32(3e38)                                   # squares past fp32's range
    x[5] = np.float32(1e-30)                                  # and below it
    y = to_host(qs.rms_norm_f32(to_dev(x), to_dev(w), 0.0)[0])
    assert np.isnan(y[1, 5]) and not np.delete(y[1], 5).any()
    assert np.isnan(y[2]).all() and np.isnan(y[3]).all()
    for i in (0, 4, 5):
        e = norm.rms_norm(x[i:i + 1], w, 0.0)[2]
        assert np.all(np.abs(y[i] - e) <= TOL * np.abs(e)), i
    (_, s), _ = qs.rms_norm_f32(to_dev(x), to_dev(w), 0.0, out_type=qs.MM_TYPE_MXFP4)
    nan = to_host(s)[:, :d // 32] == 255
    assert nan[2].all() and nan[3].all() and nan[1].sum() == 1 and not nan[[0, 4, 5]].any()


def test_graph_and_streams():
    import torch
    qs = _qs()
    say("rms_norm graph")
    x, r, w = (to_dev(v) for v in _inputs(70, 4096, 2))
    (c, s), v = qs.rms_norm_f32(x, w, residual=r, out_type=qs.MM_TYPE_F8)
    out = torch.empty_like(c), torch.empty_like(s)
    sum_out = torch.empty_like(v)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.rms_norm_f32(x, w, residual=r, out_type=qs.MM_TYPE_F8, out=out, sum_out=sum_out)
    for rep in range(3):
        for b in (*out, sum_out):
            b.view(torch.uint8).fill_(0xff)
        qs.rms_norm_f32(r, w, residual=x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0].view(torch.uint8), c.view(torch.uint8)) and torch.equal(out[1], s) and torch.equal(sum_out, v), rep
    got = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got += [qs.rms_norm_f32(x, w, residual=r)[0] for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(got[0], y) for y in got)


def test_values_past_4_gib():
    import torch
    qs = _qs()
    t, d = (1 << 18) + 5, 4128
    say("rms_norm large", t, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((t, d), device="cuda", generator=g)
    y, _ = qs.rms_norm_f32(x)
    (c, s), _ = qs.rms_norm_f32(x, out_type=qs.MM_TYPE_MXFP4)
    for at in (0, (1 << 30) // d - 4, (1 << 31) // (2 * d) - 4, t - 8):
        e = norm.rms_norm(to_host(x[at:at + 8]))[2]
        assert np.all(np.abs(to_host(y[at:at + 8]) - e) <= TOL * np.abs(e)), at
        wc, ws = qs.quantize_mxfp4(y[at:at + 8])
        assert torch.equal(c[at:at + 8], wc) and torch.equal(s[at:at + 8], ws)
