"""The e4m3 type and the mixture-of-experts layer at the sizes where offsets, grids and limits end; references in float64 on
the GPU."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import codec, f8, moe
from tests.gpu_util import say, to_dev, to_host
from tests.test_gpu_moe import ACT_EPS, sum_eps

pytestmark = pytest.mark.gpu


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


def _gen(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _values(codes):
    """float64 values of e4m3 codes on the GPU."""
    return to_dev(f8.VALUES)[codes.int()]


@pytest.mark.parametrize("rows,k,r", [((1 << 24) + 40, 128, 1), (1 << 20, 4128, 128)])
def test_quantizer_past_its_grid_and_4_gib(rows, k, r):
    """More blocks than the row quantizer has groups of lanes (2^24), values past 2^32 of the tile quantizer's input: rows
    from both ends and around each border equal the oracle's, what lies behind the outputs stays."""
    import torch
    qs = _qs()
    say("quantize_f8 large", rows, k, r)
    x = torch.randn((rows, k), device="cuda", generator=_gen(rows))
    nb, kb = -(-rows // r), -(-k // 128)
    codes = torch.full((rows * k + 64,), 0xaa, dtype=torch.uint8, device="cuda")
    scales = torch.full((nb * kb + 16,), 7.0, device="cuda")
    out = codes[:rows * k].view(rows, k), scales[:nb * kb].view(nb, kb)
    qs.quantize_f8(x, r, out=out)
    for at in (0, (1 << 24) - r if r == 1 else (1 << 32) // k // r * r, (rows - 1) // r * r):
        end = min(at + max(r, 40 if r == 1 else r), rows)
        wc, wsc = f8.quantize(to_host(x[at:end]), r)
        assert np.array_equal(to_host(out[0][at:end]), wc), at
        assert np.array_equal(to_host(out[1][at // r:at // r + len(wsc)]), wsc), at
    assert bool((codes[rows * k:] == 0xaa).all()) and bool((scales[nb * kb:] == 7).all())


@pytest.mark.parametrize("m,n", [(1, 40), (70, 130), (257, 256)])
@pytest.mark.parametrize("k", [1 << 23, (1 << 23) - 32])
def test_product_at_the_largest_k(m, n, k):
    """K = 2^23: a tile's rows span 2^31 bytes.  Bound: each block's dot of 128 products (128 steps of 2^-23 of its terms), then
    at most 4096 fused additions in a slice and 16 slices, each off by half a step of a partial sum (taken from the reference
    at every 2^18 of K, and twice that in between)."""
    import torch
    qs = _qs()
    say("f8 largest k", m, n, k)
    g = _gen(m + n)
    w = torch.randint(0, 0x7f, (n, k), dtype=torch.uint8, device="cuda", generator=g)
    w |= torch.randint(0, 2, (n, k), dtype=torch.uint8, device="cuda", generator=g) << 7
    ws = 1e-4 * (0.75 + 0.5 * torch.rand((-(-n // 128), -(-k // 128)), device="cuda", generator=g))
    x = torch.randn((m, k), device="cuda", generator=g)
    y = qs.mul_mat_f8_f32(w, ws, x)
    a, a_s = qs.quantize_f8(x)
    y8 = qs.mul_mat_f8_f8(w, ws, a, a_s)
    a, ref, mag, top = a.view(torch.uint8), 0, 0, 0
    for k0 in range(0, k, 1 << 18):
        at = slice(k0, min(k0 + (1 << 18), k))
        blocks = (torch.arange(at.start, at.stop, device="cuda")) // 128
        av = _values(a[:, at]) * a_s.double()[:, blocks]
        wv = _values(w[:, at]) * ws.double()[torch.arange(n, device="cuda") // 128][:, blocks]
        ref = ref + av @ wv.t()
        mag = mag + av.abs() @ wv.abs().t()
        top = torch.maximum(ref.abs(), torch.as_tensor(top, device="cuda", dtype=torch.float64))
    # partial sums of a slice are differences of two of the reference's
    tol = 130 * 2.0 ** -23 * mag + (4096 + 16) * 2.0 ** -23 * 4 * top
    assert bool(((y - ref).abs() <= tol).all()) and bool(((y8 - ref).abs() <= tol).all())
    assert float(tol.mean()) < 0.2 * float(ref.abs().mean())          # a wrong row would not pass


def test_product_of_more_src1_rows_than_a_grid_has_in_y():
    import torch
    qs = _qs()
    m, n, k = 70_001, 130, 160
    say("f8 many rows", m, n, k)
    g = _gen(3)
    w = torch.randint(0, 0x7f, (n, k), dtype=torch.uint8, device="cuda", generator=g)
    ws = 1e-4 * (0.75 + 0.5 * torch.rand((2, 2), device="cuda", generator=g))
    x = torch.randn((m, k), device="cuda", generator=g)
    a, a_s = qs.quantize_f8(x)
    blocks = torch.arange(k, device="cuda") // 128
    av = _values(a.view(torch.uint8)) * a_s.double()[:, blocks]
    wv = _values(w) * ws.double()[torch.arange(n, device="cuda") // 128][:, blocks]
    tol = (128 + 4 + 32) * 2.0 ** -23 * (av.abs() @ wv.abs().t())
    for y in (qs.mul_mat_f8_f32(w, ws, x), qs.mul_mat_f8_f8(w, ws, a, a_s)):
        assert bool(((y - av @ wv.t()).abs() <= tol).all())


# ---------------------------------------------------------------- the layer

def _reference(x, p, gate, up, down):
    """One expert's weights (float64, on the GPU) on tokens x with probabilities p [T, 1]: its part of dst and of the bound."""
    import torch
    c = ACT_EPS + sum_eps(max(gate.shape))
    ex = c * x.abs() + to_dev(moe.act_error(to_host(x)))
    g, u = x @ gate.t(), x @ up.t()
    eg, eu = ex @ gate.abs().t(), ex @ up.abs().t()
    s = g / (1 + torch.exp(-g))
    h = s * u
    eh = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * h.abs()
    y = h @ down.t()
    held = to_dev(moe.act_error(to_host(h.abs() + eh))) + c * (h.abs() + eh)
    return p * y, p * ((eh + held) @ down.abs().t() + 2.0 ** -20 * y.abs())


@pytest.mark.parametrize("kind,e", [("q4_0r", 140), ("f8", 80), ("f16", 40)])
def test_experts_past_4_gib(kind, e):
    """Each matrix's last expert lies past 2^32 bytes; the others are zeros, so a wrapped offset reads zeros."""
    import torch
    qs = _qs()
    d, f = 4096, 14336
    say("moe past 4 GiB", kind, e)
    g, rng = _gen(e), np.random.default_rng(e)
    mats, scales, values = [], [], []
    for n, k in ((f, d), (f, d), (d, f)):
        if kind == "q4_0r":
            q = rng.integers(0, 256, (n * k // 32, 18), dtype=np.uint8)
            q[:, :2] = (0.005 * rng.uniform(0.75, 1.25, len(q))).astype(np.float16).view(np.uint8).reshape(-1, 2)
            q = q.reshape(n, -1)
            w = torch.zeros((e, qs.repacked_bytes(n, k)), dtype=torch.uint8, device="cuda")
            w[e - 1] = qs.repack_q4_0(to_dev(q), k)
            values.append(to_dev(codec.dequantize_q4_0(q, k)).double())
        elif kind == "f8":
            w = torch.zeros((e, n, k), dtype=torch.uint8, device="cuda")
            w[e - 1] = torch.randint(0, 0x7f, (n, k), dtype=torch.uint8, device="cuda", generator=g)
            w[e - 1] |= torch.randint(0, 2, (n, k), dtype=torch.uint8, device="cuda", generator=g) << 7
            s = torch.zeros((e, n // 128, k // 128), device="cuda")
            s[e - 1] = 2e-4 * (0.75 + 0.5 * torch.rand((n // 128, k // 128), device="cuda", generator=g))
            scales.append(s)
            values.append(_values(w[e - 1]) * s[e - 1].double().repeat_interleave(128, 0).repeat_interleave(128, 1))
        else:
            w = torch.zeros((e, n, k), dtype=torch.float16, device="cuda")
            w[e - 1] = 0.03 * torch.randn((n, k), device="cuda", generator=g)
            values.append(w[e - 1].double())
        mats.append(w)
        assert w.nbytes > 1 << 32
    code = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16}[kind]
    router = torch.randn((e, d), device="cuda", generator=g) / d ** 0.5
    x = torch.randn((20, d), device="cuda", generator=g)
    x[:, 0] = 1
    router[e - 1, 0] += 20                                    # every token's first expert
    layer = qs.MoeLayer(code, router, *mats, f, 2, *scales)
    for t in (1, 3, 20):
        dst, ids, w = qs.moe_f32(layer, x[:t])
        assert bool((ids[:, 0] == e - 1).all())
        ref, err = _reference(x[:t].double(), w[:, :1].double(), *values)
        assert bool(((dst - ref).abs() <= err).all()), t
        assert float((dst - ref).norm()) <= 3e-6 * float(ref.norm()), t


@pytest.mark.parametrize("t,d,f,e,top_k", [(128, 32, 1 << 18, 16, 16), (128, 1 << 18, 32, 2, 2), (3, 1 << 18, 32, 2, 1),
                                           (1, 32, 1 << 18, 16, 16)])
def test_widest_layers(t, d, f, e, top_k):
    """Both widths at their limit: split h of 2^31 bytes with all tokens on all experts."""
    import torch
    qs = _qs()
    say("moe widest", t, d, f, e, top_k)
    g = _gen(t + e)
    mats = [(torch.randn((e, n, k), device="cuda", generator=g) / k ** 0.5).half() for n, k in ((f, d), (f, d), (d, f))]
    router = torch.randn((e, d), device="cuda", generator=g) / d ** 0.5
    x = torch.randn((t, d), device="cuda", generator=g)
    layer = qs.MoeLayer(qs.MM_TYPE_F16, router, *mats, f, top_k)
    got = qs.moe_f32(layer, x)
    dst, ids, w = got
    ri, rw = moe.select(to_host(x), to_host(router), top_k, True)
    assert np.array_equal(to_host(ids), ri) and np.all(np.abs(to_host(w) - rw) <= 2.0 ** -20 * rw)
    ref, err = torch.zeros((t, d), dtype=torch.float64, device="cuda"), torch.zeros((t, d), dtype=torch.float64, device="cuda")
    for i in range(e):
        p = to_dev(np.sum(np.where(ri == i, rw, 0), axis=1))[:, None]
        y, b = _reference(x.double(), p, *(m[i].double() for m in mats))
        ref += y
        err += b
    assert bool(((dst - ref).abs() <= err).all())
    assert float((dst - ref).norm()) <= 1e-5 * float(ref.norm())
    assert all(torch.equal(a, b) for a, b in zip(got, qs.moe_f32(layer, x)))
