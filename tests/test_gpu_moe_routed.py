"""GPU parity of the experts for a given routing, of MXFP4 experts, and of a run of the operators as a decoder uses them."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import codec, f8, moe, mx4, norm, route
from tests.gpu_util import say, to_dev, to_host
from tests.test_gpu_moe import ACT_EPS, sum_eps

pytestmark = pytest.mark.gpu


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


class Layer:
    """Random experts of one kind: their values in float64 and the library's layer, without a router or with one."""

    def __init__(self, kind, d, f, e, top_k, seed, router=False):
        import torch
        qs = _qs()
        rng = np.random.default_rng(seed)
        self.values, dev, scales = [], [], []
        for n, k in ((f, d), (f, d), (d, f)):
            w = (rng.standard_normal((e, n, k)) * 0.05).astype(np.float32)
            if kind == "q4_0r":
                q = [codec.quantize_q4_0(v) for v in w]
                self.values.append(np.stack([codec.dequantize_q4_0(v, k) for v in q]).astype(np.float64))
                dev.append(torch.stack([qs.repack_q4_0(to_dev(v), k) for v in q]))
                scales.append(None)
            elif kind == "f16":
                self.values.append(w.astype(np.float16).astype(np.float64))
                dev.append(to_dev(w.astype(np.float16)))
                scales.append(None)
            else:
                q = [f8.quantize(v, 128) if kind == "f8" else mx4.quantize(v) for v in w]
                self.values.append(np.stack([f8.dequantize(*v, 128) if kind == "f8" else mx4.dequantize(*v) for v in q]))
                dev.append(to_dev(np.stack([c for c, _ in q])))
                s = np.stack([s for _, s in q])
                if kind == "mxfp4":
                    s[:, :, k // 32:] = 255                   # padding: not to be read
                scales.append(to_dev(s))
        self.code = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16, "mxfp4": qs.MM_TYPE_MXFP4}[kind]
        self.dev, self.scales, self.f, self.top_k = dev, scales, f, top_k
        self.router = (rng.standard_normal((e, d)) / np.sqrt(d)).astype(np.float32) if router else None
        self.layer = qs.MoeLayer(self.code, to_dev(self.router) if router else None, *dev, f, top_k, *scales, d=d)

    def oracle(self, x, ids, w):
        """dst and a bound of |dst - exact|, as oracle.moe.layer's, for a choice that is given."""
        gate, up, down = self.values
        e = gate.shape[0]
        x = x.astype(np.float64)
        dst, err = np.zeros_like(x), np.zeros_like(x)
        c = ACT_EPS + sum_eps(max(gate.shape[1:]))
        for t in range(x.shape[0]):
            for j in range(ids.shape[1]):
                i, p = ids[t, j], float(w[t, j])
                if not 0 <= i < e:
                    continue
                g, u = gate[i] @ x[t], up[i] @ x[t]
                ex = c * np.abs(x[t]) + moe.act_error(x[t])
                eg, eu = np.abs(gate[i]) @ ex, np.abs(up[i]) @ ex
                s = g / (1 + np.exp(-g))
                h = s * u
                eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * 2.0 ** -24 * np.abs(h)
                y = down[i] @ h
                held = c * (np.abs(h) + eh) + moe.act_error(np.abs(h) + eh)
                dst[t] += p * y
                err[t] += abs(p) * (np.abs(down[i]) @ (eh + held) + 2.0 ** -20 * np.abs(y))
        return dst, err

    def check(self, x, ids, w, what=""):
        qs = _qs()
        dst = to_host(qs.moe_routed_f32(self.layer, to_dev(x), to_dev(ids), to_dev(w)))
        ref, err = self.oracle(x, ids, w)
        assert np.all(np.abs(dst - ref) <= err), f"{what}: {np.nanmax(np.abs(dst - ref) / err):.3g} of the bound"
        return dst


def _choice(rng, t, e, k):
    ids = np.stack([rng.permutation(e)[:k] for _ in range(t)]).astype(np.int32)
    return ids, rng.uniform(0.1, 1, (t, k)).astype(np.float32)


def _x(rng, t, d):
    x = rng.standard_normal((t, d)).astype(np.float32)
    x[:, rng.random(d) < 0.02] *= 10
    return x


KINDS = ["mxfp4", "q4_0r", "f8", "f16"]


ROUTED = [
    (1, 256, 128, 4, 2), (1, 32, 32, 1, 1), (1, 2080, 1056, 12, 3), (2, 288, 160, 5, 5), (7, 416, 96, 12, 3),
    (16, 512, 256, 8, 2), (17, 256, 288, 3, 1), (24, 512, 1024, 2, 2), (33, 160, 64, 40, 8), (32, 512, 1024, 2, 2),
    (64, 128, 96, 2, 2), (100, 96, 128, 16, 4), (128, 64, 32, 512, 16),
    # few tokens, on both sides of what the gate / up kernel holds of x
    (1, 8192, 64, 3, 2), (1, 8224, 64, 3, 2), (2, 4096, 96, 5, 3), (4, 2048, 64, 16, 16), (4, 2080, 64, 6, 4), (3, 2752, 64, 4, 2),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,d,f,e,top_k", ROUTED)
def test_routed(kind, t, d, f, e, top_k):
    say("moe routed", kind, t, d, f, e, top_k)
    m = Layer(kind, d, f, e, top_k, t * 100 + d + f + e)
    rng = np.random.default_rng(t + e)
    m.check(_x(rng, t, d), *_choice(rng, t, e, top_k), what=f"{kind} T={t} D={d} F={f} E={e} k={top_k}")


# the shapes of the layer with its own router: rows of gate / up walked, all output tiles, slices of down
WITH_ROUTER = [
    (1, 256, 128, 4, 2), (1, 2080, 1056, 12, 3), (4, 160, 8256, 8, 2), (16, 160, 4128, 16, 2), (24, 512, 8192, 2, 2), (33, 160, 64, 40, 8),
    (40, 96, 33024, 2, 2), (70, 96, 16416, 2, 2), (128, 64, 32, 512, 16),
]


@pytest.mark.parametrize("t,d,f,e,top_k", WITH_ROUTER)
def test_mxfp4_experts_with_a_router(t, d, f, e, top_k):
    say("moe mxfp4", t, d, f, e, top_k)
    qs = _qs()
    m = Layer("mxfp4", d, f, e, top_k, t + d + f, router=True)
    x = _x(np.random.default_rng(t), t, d)
    got = qs.moe_f32(m.layer, to_dev(x))
    dst, ids, w = (to_host(v) for v in got)
    ri, rw = moe.select(x, m.router, top_k, True)
    assert np.array_equal(ids, ri) and np.all(np.abs(w - rw) <= 2.0 ** -20 * rw)
    ref, err = m.oracle(x, ri, rw)
    assert np.all(np.abs(dst - ref) <= err) and np.linalg.norm(dst - ref) <= 3e-6 * np.linalg.norm(ref)
    assert all(np.array_equal(to_host(a), to_host(b)) for a, b in zip(got, qs.moe_f32(m.layer, to_dev(x))))
    # the same choice given: the same products, in the same order
    assert np.array_equal(to_host(qs.moe_routed_f32(m.layer, to_dev(x), got[1], got[2])), dst)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [1, 3, 20])
def test_slots_without_an_expert(kind, t):
    """Ids out of range add nothing, whatever their weight; a token without experts gets zeros."""
    say("moe routed empty slots", kind, t)
    m = Layer(kind, 160, 96, 6, 4, t)
    rng = np.random.default_rng(t)
    x = _x(rng, t, 160)
    ids, w = _choice(rng, t, 6, 4)
    bad = np.array([-1, 6, np.iinfo(np.int32).min, np.iinfo(np.int32).max, 65535, 512, 1 << 16], np.int32)
    for i in range(t):
        ids[i, rng.permutation(4)[:rng.integers(1, 4)]] = rng.choice(bad)
    w[(ids < 0) | (ids >= 6)] = np.nan
    m.check(x, ids, w, kind)
    ids[0] = -1
    dst = m.check(x, ids, w, kind)
    assert not dst[0].any()
    ids[:] = bad[rng.integers(0, len(bad), ids.shape)]
    assert not m.check(x, ids, w, kind).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,top_k", [(1, 3), (5, 8), (40, 4), (128, 8)])
def test_an_expert_named_several_times(kind, t, top_k):
    say("moe routed twice", kind, t, top_k)
    m = Layer(kind, 96, 64, 9, top_k, t + top_k)
    rng = np.random.default_rng(t)
    x = _x(rng, t, 96)
    ids = rng.integers(0, 3, (t, top_k)).astype(np.int32)
    ids[-1] = 8                                               # all of a token's slots
    w = rng.uniform(-1, 1, (t, top_k)).astype(np.float32)
    once_i, once_w = np.full_like(ids, -1), np.zeros((t, top_k))
    for i in range(t):
        for j, e in enumerate(dict.fromkeys(ids[i])):
            once_i[i, j], once_w[i, j] = e, w[i].astype(np.float64)[ids[i] == e].sum()
    qs = _qs()
    got = to_host(qs.moe_routed_f32(m.layer, to_dev(x), to_dev(ids), to_dev(w)))
    ref, err = m.oracle(x, once_i, once_w)
    # the sum of up to top_k weights in fp32: half a step of the magnitudes' sum each
    mags = np.zeros_like(ref)
    for i in range(t):
        for j in range(top_k):
            if once_i[i, j] >= 0:
                one, _ = m.oracle(x[i:i + 1], once_i[i:i + 1, j:j + 1], np.ones((1, 1)))
                mags[i] += np.abs(one[0]) * np.abs(w[i])[ids[i] == once_i[i, j]].sum()
    assert np.all(np.abs(got - ref) <= err + top_k * 2.0 ** -24 * mags)


@pytest.mark.parametrize("kind", KINDS)
def test_nan_reaches_its_token_only(kind):
    say("moe routed nan", kind)
    qs = _qs()
    m = Layer(kind, 96, 64, 5, 2, 3)
    rng = np.random.default_rng(1)
    x = _x(rng, 21, 96)
    ids, w = _choice(rng, 21, 5, 2)
    ref, err = m.oracle(x, ids, w)
    x[2, 7], x[9, 95], w[4, 1] = np.nan, np.inf, np.nan
    dst = to_host(qs.moe_routed_f32(m.layer, to_dev(x), to_dev(ids), to_dev(w)))
    bad = [2, 4, 9]
    assert np.isnan(dst[bad]).all()
    good = np.setdiff1d(np.arange(21), bad)
    assert np.all(np.abs(dst[good] - ref[good]) <= err[good])


def test_nan_block_of_an_expert_that_is_not_used():
    qs = _qs()
    say("moe mxfp4 nan expert")
    m = Layer("mxfp4", 96, 64, 4, 2, 8)
    rng = np.random.default_rng(8)
    x, ids = _x(rng, 5, 96), np.tile(np.array([[0, 2]], np.int32), (5, 1))
    ids[3, 1] = 1
    w = np.ones((5, 2), np.float32)
    for s in m.scales:
        s[1, 3, 0] = 255
    dst = to_host(qs.moe_routed_f32(m.layer, to_dev(x), to_dev(ids), to_dev(w)))
    assert np.isnan(dst[3]).any() and np.isfinite(np.delete(dst, 3, axis=0)).all()


@pytest.mark.parametrize("t", [1, 5, 60])
def test_smallest_scales_of_experts(t):
    """Scale bytes 0 (2^-127, below fp32's normal range), 1 and 2 in gate and up, with activations of about 2^100."""
    say("moe mxfp4 smallest scales", t)
    m = Layer("mxfp4", 160, 96, 3, 2, 5)
    rng = np.random.default_rng(t)
    for i in (0, 1):
        codes, scales = to_host(m.dev[i]), to_host(m.scales[i])
        scales[:, :, :5] = rng.integers(0, 3, scales[:, :, :5].shape)
        m.scales[i].copy_(to_dev(scales))
        m.values[i] = np.stack([mx4.dequantize(c, s) for c, s in zip(codes, scales)])
    x = _x(rng, t, 160) * np.float32(2.0 ** 100)
    dst = m.check(x, *_choice(rng, t, 3, 2))
    assert (np.abs(dst) > 0).mean() > 0.99


@pytest.mark.parametrize("kind", ["mxfp4", "f16"])
@pytest.mark.parametrize("t", [1, 6, 40])
def test_graph_replays_follow_their_inputs(kind, t):
    import torch
    qs = _qs()
    say("moe routed graph", kind, t)
    m = Layer(kind, 160, 128, 12, 3, 4)
    rng = np.random.default_rng(t)
    cases = [(_x(rng, t, 160), *_choice(rng, t, 12, 3)) for _ in range(3)]
    dev = [[to_dev(v) for v in c] for c in cases]
    want = [qs.moe_routed_f32(m.layer, *c) for c in dev]
    x, ids, w = (v.clone() for v in dev[0])
    out = torch.empty_like(want[0])
    ws = torch.empty(m.layer.routed_workspace_size(t), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qs.moe_routed_f32(m.layer, x, ids, w, out=out, ws=ws)
    for c, y in zip(dev[::-1], want[::-1]):
        for to, v in zip((x, ids, w), c):
            to.copy_(v)
        ws.fill_(0xff)
        qs.moe_routed_f32(m.layer, *dev[1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
        assert torch.equal(ids, c[1]) and torch.equal(w, c[2])


@pytest.mark.parametrize("t", [2, 20])
def test_two_streams_at_once(t):
    """Routing and experts on two streams, inputs of their own, workspaces of their own: the bits of one after the other."""
    import torch
    qs = _qs()
    say("moe routed two streams", t)
    m = Layer("mxfp4", 256, 512, 12, 3, 9)
    rng = np.random.default_rng(t)
    router = qs.Router(12, 3)
    xs = [to_dev(_x(rng, t, 256)) for _ in range(2)]
    logits = [to_dev(rng.standard_normal((t, 12)).astype(np.float32)) for _ in range(2)]
    want = [qs.moe_routed_f32(m.layer, x, *qs.route_f32(router, l)) for x, l in zip(xs, logits)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(qs.moe_routed_f32(m.layer, xs[i], *qs.route_f32(router, logits[i])))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_mxfp4_experts_past_4_gib():
    """The last expert of each matrix lies past 2^32 bytes."""
    import torch
    qs = _qs()
    d, f, e = 4096, 14336, 150
    say("moe mxfp4 past 4 GiB", e)
    g = torch.Generator(device="cuda")
    g.manual_seed(e)
    mats, scales, values = [], [], []
    for n, k in ((f, d), (f, d), (d, f)):
        w = torch.zeros((e, n, k // 2), dtype=torch.uint8, device="cuda")
        s = torch.full((e, n, k // 32), 127, dtype=torch.uint8, device="cuda")
        w[e - 1] = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        s[e - 1] = torch.randint(118, 121, (n, k // 32), dtype=torch.uint8, device="cuda", generator=g)
        assert w.nbytes > 1 << 32
        mats.append(w)
        scales.append(s)
        values.append(qs.dequantize_mxfp4(w[e - 1], s[e - 1]).double())
    layer = qs.MoeLayer(qs.MM_TYPE_MXFP4, None, *mats, f, 2, *scales)
    x = torch.randn((20, d), device="cuda", generator=g)
    ids = torch.tensor([[0, e - 1]], dtype=torch.int32, device="cuda").repeat(20, 1)
    w = torch.full((20, 2), 0.5, device="cuda")
    for t in (1, 3, 20):
        dst = qs.moe_routed_f32(layer, x[:t], ids[:t], w[:t])
        gate, up = x[:t].double() @ values[0].t(), x[:t].double() @ values[1].t()
        ref = 0.5 * (gate / (1 + torch.exp(-gate)) * up) @ values[2].t()
        assert float((dst - ref).norm()) <= 3e-6 * float(ref.norm()), t


def test_a_step_of_a_decoder():
    """Norm with the residual, MXFP4 product, norm, router product, routing, experts, as one run and as a captured one: each
    operator's output against its oracle on the inputs it had, and the same bits on every replay."""
    import torch
    qs = _qs()
    say("decoder step")
    t, d, f, e, k = 5, 512, 256, 16, 4
    rng = np.random.default_rng(11)
    m = Layer("mxfp4", d, f, e, k, 6)
    h0, r0 = _x(rng, t, d), _x(rng, t, d)
    g1, g2 = (1 + 0.1 * rng.standard_normal((2, d))).astype(np.float32)
    proj, ps = mx4.quantize((0.05 * rng.standard_normal((d, d))).astype(np.float32))
    wr = (rng.standard_normal((e, d)) / np.sqrt(d)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(e)).astype(np.float32)
    h, r, g1d, g2d, pd, psd, wrd = (to_dev(v) for v in (h0, r0, g1, g2, proj, ps, wr))
    router = qs.Router(e, k, score="sigmoid", bias=to_dev(bias), groups=4, group_k=2, group_top=2, scale=1.5)

    def step(h, r):
        a, v1 = qs.rms_norm_f32(h, g1d, residual=r, out_type=qs.MM_TYPE_MXFP4)
        y = qs.mul_mat_mxfp4_mxfp4(pd, psd, *a)
        n, v2 = qs.rms_norm_f32(y, g2d, residual=v1)
        logits = qs.mul_mat_f32(wrd, n)
        ids, w = qs.route_f32(router, logits)
        return a, v1, y, n, v2, logits, ids, w, qs.moe_routed_f32(m.layer, n, ids, w)

    got = step(h, r)
    (ac, as_), v1, y, n, v2, logits, ids, w, dst = ([to_host(q) for q in v] if isinstance(v, tuple) else to_host(v) for v in got)
    y1, s1, _ = norm.rms_norm(h0, g1, 1e-5, r0)
    wc, wsc = mx4.quantize(y1)
    assert np.array_equal(v1, s1) and np.array_equal(ac, wc) and np.array_equal(as_, wsc)
    ref, mag = mx4.mul_mat(proj, ps, ac, as_)
    assert np.all(np.abs(y - ref) <= 2.0 ** -19 * mag)
    _, s2, exact = norm.rms_norm(y, g2, 1e-5, v1)
    assert np.array_equal(v2, s2) and np.all(np.abs(n - exact) <= 3.01 * 2.0 ** -24 * np.abs(exact))
    ri, rw = route.route(logits, k, score="sigmoid", bias=bias, groups=4, group_k=2, group_top=2, scale=1.5)
    assert np.array_equal(ids, ri) and np.all(np.abs(w - rw) <= 2.0 ** -23 * rw)
    ref, err = m.oracle(n, ids, w)
    assert np.all(np.abs(dst - ref) <= err)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(h, r)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(h, r)[-1]
    for _ in range(3):
        out.fill_(float("nan"))
        step(r, h)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_host(out), dst)
