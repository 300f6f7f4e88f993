"""GPU parity of the mixture-of-experts layer against the float64 oracle: chosen experts equal, weights and dst
within the bound that its roundings allow."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import codec, f8, moe
from tests.gpu_util import say, to_dev, to_host

pytestmark = pytest.mark.gpu

ACT_EPS = 2.0 ** -21      # 22 significant bits relative to the block, with the power of two's slack


def sum_eps(k):
    """Sum of k exact products in fp32: 32 per block and its two parts, each addition off by at most one step
    (2^-23), a scale product and an fma per block, the join of 8 waves."""
    return (64 + 2 * (k // 32) + 16) * 2.0 ** -23


def _qs():
    import quantized_skinny_gemm_amd as qs
    return qs


class Layer:
    def __init__(self, kind, t, d, f, e, top_k, seed, norm=True):
        import torch
        qs = _qs()
        rng = np.random.default_rng(seed)
        self.kind, self.top_k, self.norm = kind, top_k, norm
        self.x = rng.standard_normal((t, d)).astype(np.float32)
        self.x[:, rng.random(d) < 0.02] *= 10
        self.router = (rng.standard_normal((e, d)) / np.sqrt(d)).astype(np.float32)
        self.values, dev, scales = [], [], []
        for n, k in ((f, d), (f, d), (d, f)):
            w = (rng.standard_normal((e, n, k)) * 0.05).astype(np.float32)
            if kind == "q4_0r":
                q = [codec.quantize_q4_0(v) for v in w]
                self.values.append(np.stack([codec.dequantize_q4_0(v, k) for v in q]).astype(np.float64))
                dev.append(torch.stack([qs.repack_q4_0(to_dev(v), k) for v in q]))
                scales.append(None)
            elif kind == "f8":
                q = [f8.quantize(v, 128) for v in w]
                self.values.append(np.stack([f8.dequantize(c, s, 128) for c, s in q]))
                dev.append(to_dev(np.stack([c for c, _ in q])))
                scales.append(to_dev(np.stack([s for _, s in q])))
            else:
                self.values.append(w.astype(np.float16).astype(np.float64))
                dev.append(to_dev(w.astype(np.float16)))
                scales.append(None)
        code = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16}[kind]
        self.dev = dev
        self.layer = qs.MoeLayer(code, to_dev(self.router), *dev, f, top_k, *scales, norm=norm)

    def oracle(self, x=None):
        x = self.x if x is None else x
        d, f = self.values[0].shape[2], self.values[0].shape[1]
        return moe.layer(x, self.router, *self.values, self.top_k, self.norm, ACT_EPS, sum_eps(max(d, f)))

    def check(self, got, x=None, what=""):
        dst, ids, w = (to_host(v) for v in got)
        rd, ri, rw, err = self.oracle(x)
        assert np.array_equal(ids, ri), what
        assert np.all(np.abs(w - rw) <= 2.0 ** -20 * rw), what
        assert np.all(np.abs(dst - rd) <= err), f"{what}: {np.max(np.abs(dst - rd) / err):.3g} of the bound"
        # and no more than the fp32 sums' own noise in the mean
        assert np.linalg.norm(dst - rd) <= 3e-6 * np.linalg.norm(rd), what


KINDS = ["q4_0r", "f8", "f16"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,d,f,e,top_k", [
    (1, 256, 128, 4, 2), (1, 32, 32, 1, 1), (1, 2080, 1056, 12, 3), (2, 288, 160, 5, 5), (7, 416, 96, 12, 3),
    (16, 512, 256, 8, 2), (17, 256, 288, 3, 1), (33, 160, 64, 40, 8), (64, 128, 96, 2, 2), (100, 96, 128, 16, 4),
    (128, 64, 32, 512, 16),
])
def test_layer(kind, t, d, f, e, top_k):
    say("moe", kind, t, d, f, e, top_k)
    m = Layer(kind, t, d, f, e, top_k, t * 100 + d + f + e)
    qs = _qs()
    m.check(qs.moe_f32(m.layer, to_dev(m.x)), what=f"{kind} T={t} D={d} F={f} E={e} k={top_k}")


# many row groups: a workgroup of gate / up walks several of them, with one to three passes over the tokens
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,d,f,e,top_k", [
    (16, 160, 4128, 16, 2), (4, 160, 8256, 8, 2), (1, 1056, 8256, 4, 4), (40, 96, 33024, 2, 2),
])
def test_layer_walks_row_groups(kind, t, d, f, e, top_k):
    say("moe wide", kind, t, d, f, e, top_k)
    m = Layer(kind, t, d, f, e, top_k, t + d + f + e)
    qs = _qs()
    got = qs.moe_f32(m.layer, to_dev(m.x))
    m.check(got, what=f"{kind} T={t} D={d} F={f} E={e} k={top_k}")
    assert all(np.array_equal(to_host(a), to_host(b)) for a, b in zip(got, qs.moe_f32(m.layer, to_dev(m.x))))


@pytest.mark.parametrize("kind", KINDS)
def test_probabilities_without_normalisation(kind):
    say("moe no norm", kind)
    m = Layer(kind, 5, 256, 96, 10, 3, 77, norm=False)
    m.check(_qs().moe_f32(m.layer, to_dev(m.x)), what=kind)


def test_ties_take_the_lower_index():
    import torch
    qs = _qs()
    say("moe ties")
    m = Layer("f16", 3, 64, 32, 70, 4, 5)
    m.router[:] = 0
    m.router[33] = m.router[65] = m.router[69] = m.x[0] * 0.01
    m.layer = qs.MoeLayer(qs.MM_TYPE_F16, to_dev(m.router), *m.dev, 32, 4)
    _, ids, _ = qs.moe_f32(m.layer, to_dev(m.x))
    assert to_host(ids)[0].tolist() == [33, 65, 69, 0]
    _, ri, _, _ = m.oracle()
    assert np.array_equal(to_host(ids), ri)
    assert ids.dtype == torch.int32


@pytest.mark.parametrize("kind", KINDS)
def test_all_tokens_on_one_expert_and_scale_range(kind):
    """128 tokens that all take the same two experts (several passes of 16), activations from 2^-30 to 2^12."""
    say("moe one expert", kind)
    qs = _qs()
    m = Layer(kind, 128, 96, 64, 9, 2, 31)
    m.x = np.abs(m.x) * (2.0 ** np.linspace(-30, 6, 128))[:, None].astype(np.float32)
    m.router = np.abs(m.router)
    m.router[4] += 1
    m.router[7] += 2
    m.layer = qs.MoeLayer(m.layer.struct.type, to_dev(m.router), *m.dev, 64, 2, *m.layer.tensors[4:])
    got = qs.moe_f32(m.layer, to_dev(m.x.astype(np.float32)))
    assert np.array_equal(to_host(got[1])[-1], [7, 4])
    dst, ids, _ = (to_host(v) for v in got)
    rd, ri, _, err = m.oracle()
    assert np.array_equal(ids, ri) and np.all(np.abs(dst - rd) <= err)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [3, 40])
def test_non_finite_values_stay_in_their_token(kind, t):
    """A NaN token, an infinite token, and a NaN in a weight of one expert: NaN for the tokens concerned, the other
    rows as the oracle has them; ids stay valid."""
    import torch
    say("moe nan", kind, t)
    qs = _qs()
    m = Layer(kind, t, 160, 96, 6, 2, 91)
    x = m.x.copy()
    x[0, 3] = np.nan
    x[1, 100] = np.inf
    dst, ids, w = qs.moe_f32(m.layer, to_dev(x))
    y, i = to_host(dst), to_host(ids)
    assert np.isnan(y[:2]).all() and np.isfinite(y[2:]).all()
    assert ((i >= 0) & (i < 6)).all()
    rd, ri, _, err = m.oracle()
    assert np.all(np.abs(y[2:] - rd[2:]) <= err[2:])
    if kind != "q4_0r":
        bad = int(ri[2, 0])
        m.dev[2][bad].view(torch.uint8)[5].fill_(0x7f)          # row 5 of down: NaN in both types
        y = to_host(qs.moe_f32(m.layer, to_dev(m.x))[0])
        uses = (ri == bad).any(axis=1)
        assert np.isnan(y[uses][:, 5]).all()
        ok = np.ones_like(y, bool)
        ok[uses, 5] = False
        assert np.isfinite(y[ok]).all() and np.all(np.abs(y - rd)[ok] <= err[ok])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", [1, 20])
def test_graph_streams_and_rows_behind_the_batch(kind, t):
    """Replays of a captured call with eager work between them, two streams with their own workspaces, out-buffers
    longer than the batch: the same bits, and nothing else written."""
    import torch
    say("moe graph", kind, t)
    qs = _qs()
    m = Layer(kind, t, 256, 160, 8, 3, 13)
    x = to_dev(m.x)
    want = [v.clone() for v in qs.moe_f32(m.layer, x)]
    m.check(want, what="eager")
    buf = torch.full((t + 1, 256), 7.0, device="cuda")
    ids = torch.full((t + 1, 3), -5, dtype=torch.int32, device="cuda")
    w = torch.full((t + 1, 3), 7.0, device="cuda")
    ws = torch.full((m.layer.workspace_size(t),), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qs.moe_f32(m.layer, x, out=buf[:t], ids=ids[:t], weights=w[:t], ws=ws)
    for rep in range(3):
        buf[:t] = float("nan")
        ws.fill_(0xff)
        qs.moe_f32(m.layer, x * 3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf[:t], want[0]) and torch.equal(ids[:t], want[1]) and torch.equal(w[:t], want[2]), rep
    assert bool((buf[t] == 7).all()) and bool((ids[t] == -5).all()) and bool((w[t] == 7).all())
    got = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append([qs.moe_f32(m.layer, x)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[0]) for ys in got for y in ys)


@pytest.mark.parametrize("kind", KINDS)
def test_much_used_experts_give_the_same_bits_every_time(kind):
    """128 tokens on 4 experts, top 2 (about 64 tokens an expert, several jobs each): eight calls, one result."""
    import torch
    say("moe determinism", kind)
    qs = _qs()
    m = Layer(kind, 128, 256, 288, 4, 2, 3)
    x = to_dev(m.x)
    want = qs.moe_f32(m.layer, x)[0].clone()
    m.check(qs.moe_f32(m.layer, x), what=kind)
    for _ in range(7):
        assert torch.equal(qs.moe_f32(m.layer, x)[0], want)


def test_decode_step_quantize_project_route_and_project_again():
    """The operators as a decode step uses them: projections with e4m3 weights on an activation quantized once,
    the layer with e4m3 experts, the output projection; against the float64 composition."""
    say("decode step f8")
    qs = _qs()
    rng = np.random.default_rng(8)
    m = Layer("f8", 4, 256, 160, 8, 2, 21)
    wq, wqs = f8.quantize((rng.standard_normal((256, 256)) * 0.06).astype(np.float32), 128)
    wo, wos = f8.quantize((rng.standard_normal((500, 256)) * 0.06).astype(np.float32), 128)
    a, a_s = qs.quantize_f8(to_dev(m.x), 1)
    q = qs.mul_mat_f8_f8(to_dev(wq), to_dev(wqs), a, a_s)
    x1 = to_host(q)
    y, ids, w = qs.moe_f32(m.layer, q)
    m.check((y, ids, w), x=x1, what="layer in the step")
    logits = to_host(qs.mul_mat_f8_f32(to_dev(wo), to_dev(wos), y))
    b, b_s = f8.quantize(to_host(y), 1)
    ref, mag = f8.mul_mat(wo, wos, b, b_s)
    assert np.all(np.abs(logits - ref) <= (128 + 4 + 32) * 2.0 ** -23 * mag)
    ra, ras = f8.quantize(m.x, 1)
    ref, mag = f8.mul_mat(wq, wqs, ra, ras)
    assert np.all(np.abs(x1 - ref) <= (128 + 4 + 32) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("exponent", [-30, -54, -58])
def test_small_activations_keep_their_bits(kind, exponent):
    """Activations of about 2^exponent (h of about its square, dst down to 1e-38, nearly all in fp32's normal range):
    as accurate as at unit scale, also where only the expert with a weight near 2^-10 adds to dst."""
    say("moe small", kind, exponent)
    qs = _qs()
    m = Layer(kind, 3, 256, 128, 2, 2, 11)
    m.x = (m.x * np.float32(2.0 ** exponent)).astype(np.float32)
    m.check(qs.moe_f32(m.layer, to_dev(m.x)), what=f"{kind} 2^{exponent}")
    m.x[:, 7] = np.float32(2.0 ** exponent)
    m.router[0] = m.router[1]
    m.router[1, 7] += np.float32(2.0 ** -exponent * 7)        # weights 1 / (1 + e^-7) and e^-7 / (1 + e^-7)
    m.dev[2][1].zero_()                                       # zeros are the value 0 in every type
    m.values[2][1] = 0
    m.layer = qs.MoeLayer(m.layer.struct.type, to_dev(m.router), *m.dev, 128, 2, *m.layer.tensors[4:])
    got = qs.moe_f32(m.layer, to_dev(m.x))
    assert got[1].tolist() == [[1, 0]] * 3 and bool((got[2][:, 1] < 2.0 ** -9).all())
    m.check(got, what=f"{kind} 2^{exponent}, small weight")


@pytest.mark.parametrize("kind", KINDS)
def test_layer_reads_the_storage_that_its_weights_have_now(kind):
    import torch
    say("moe new storage", kind)
    qs = _qs()
    m, other = Layer(kind, 5, 128, 96, 4, 2, 61), Layer(kind, 5, 128, 96, 4, 2, 62)
    x = to_dev(m.x)
    qs.moe_f32(m.layer, x)
    torch.cuda.synchronize()
    for mine, new in zip(m.layer.tensors, other.layer.tensors):
        if mine is not None:
            mine.data = new.clone()
    m.values, m.router = other.values, other.router
    m.check(qs.moe_f32(m.layer, x), what=kind)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("t,e", [(1, 6), (5, 6), (40, 64)])
def test_infinite_logits(t, e, norm):
    """Minus infinity masks an expert (probability 0, chosen last), also where fewer than top_k are left; plus infinity,
    or nothing but minus infinity, makes the token NaN; ids stay valid."""
    say("moe infinite logits", t, e, norm)
    qs = _qs()
    m = Layer("f16", t, 96, 64, e, 2, 17, norm=norm)
    m.x[:, 0] = 1
    if t > 1:
        m.x[1, 0] = -1                                        # plus infinity where the others have minus
    router = m.router.copy()

    def run(masked):
        m.router = router.copy()
        m.router[masked, 0] = -np.inf
        m.layer = qs.MoeLayer(qs.MM_TYPE_F16, to_dev(m.router), *m.dev, 64, 2, norm=norm)
        return [to_host(v) for v in qs.moe_f32(m.layer, to_dev(m.x))]

    good = [i for i in range(t) if i != 1]
    best = np.argmax(m.x.astype(np.float64) @ router.T.astype(np.float64), axis=1)
    for masked in ([int(best[0])], list(range(e - 1)), [0]):
        dst, ids, w = run(masked)
        with np.errstate(invalid="ignore"):                   # token 1
            rd, ri, rw, err = m.oracle()
        assert np.array_equal(ids[good], ri[good])
        assert np.all(np.abs(w - rw)[good] <= 2.0 ** -20 * rw[good]) and np.all(np.abs(dst - rd)[good] <= err[good])
        assert np.all(w[good][np.isin(ids[good], masked)] == 0)
        if t > 1:
            assert np.isnan(dst[1]).all() and np.isnan(w[1]).all() and ids[1, 0] == min(masked)
    dst, ids, w = run(list(range(e)))
    assert np.isnan(dst).all() and np.isnan(w).all() and np.array_equal(ids, [[0, 1]] * t)


@pytest.mark.parametrize("t", [1, 7, 20])
def test_values_far_below_their_blocks_largest(t):
    """Activations of 2^-27 of the one large value of their block, which meets zero weights: what is kept of them
    decides the result.  2^-27 + 0.98 * 2^-39 is held as 2^-27 (the bound's worst case), and all weights are positive,
    so that these errors add up: past a bound that is relative to each value, within the one that holds."""
    say("moe far below", t)
    qs = _qs()
    m = Layer("f16", t, 64, 32, 2, 1, 41)
    m.x[:] = np.float32(2.0 ** -27 + 0.98 * 2.0 ** -39)
    m.x[:, ::32] = 1
    for w, v in zip(m.dev, m.values):
        w.abs_()
        np.abs(v, out=v)
    for i in (0, 1):
        m.dev[i][:, :, ::32] = 0
        m.values[i][:, :, ::32] = 0
    dst, ids, _ = (to_host(v) for v in qs.moe_f32(m.layer, to_dev(m.x)))
    rd, ri, _, err = m.oracle()
    assert np.array_equal(ids, ri) and np.all(np.abs(dst - rd) <= err)
    assert np.all(np.abs(dst - rd) > 2.0 ** -13 * rd)


# A layer whose waves take several units of K in a row group and several row groups, and whose down is cut in slices;
# (T, plan of each kind as rt, slices), held to the plans by tests/test_f8_moe_host.py.
LONG = dict(d=2112, f=16416, e=2, top_k=2)
LONG_PLANS = {3: {"q4_0r": (1, 1), "f8": (1, 1), "f16": (1, 1)}, 7: {"q4_0r": (4, 4), "f8": (2, 4), "f16": (4, 4)},
              16: {"q4_0r": (4, 4), "f8": (2, 4), "f16": (4, 4)}, 24: {"q4_0r": (4, 4), "f8": (2, 4), "f16": (4, 4)},
              40: {"q4_0r": (2, 4), "f8": (1, 1), "f16": (2, 4)}, 100: {"q4_0r": (1, 1), "f8": (1, 1), "f16": (1, 1)}}


class LongLayer:
    """Random codes and scales; the float64 values are on the GPU, where the reference is computed."""

    def __init__(self, kind):
        import torch
        qs = _qs()
        d, f, e, k = (LONG[n] for n in ("d", "f", "e", "top_k"))
        rng = np.random.default_rng(97)
        self.values, dev, scales = [], [], []
        for n, width in ((f, d), (f, d), (d, f)):
            if kind == "q4_0r":
                q = rng.integers(0, 256, (e * n * width // 32, 18), dtype=np.uint8)
                q[:, :2] = (0.01 * rng.uniform(0.75, 1.25, len(q))).astype(np.float16).view(np.uint8).reshape(-1, 2)
                q = q.reshape(e, n, -1)
                values = np.stack([codec.dequantize_q4_0(v, width) for v in q])
                dev.append(torch.stack([qs.repack_q4_0(to_dev(v), width) for v in q]))
                scales.append(None)
            elif kind == "f8":
                c = rng.integers(0, 0x7f, (e, n, width), dtype=np.uint8) | (rng.integers(0, 2, (e, n, width), dtype=np.uint8) << 7)
                s = (4e-4 * rng.uniform(0.75, 1.25, (e, -(-n // 128), -(-width // 128)))).astype(np.float32)
                values = np.stack([f8.dequantize(c[i], s[i], 128) for i in range(e)])
                dev.append(to_dev(c))
                scales.append(to_dev(s))
            else:
                values = (rng.standard_normal((e, n, width), dtype=np.float32) * 0.05).astype(np.float16)
                dev.append(to_dev(values))
                scales.append(None)
            self.values.append(to_dev(values).double())
        self.x = rng.standard_normal((100, d)).astype(np.float32)
        self.router = (rng.standard_normal((e, d)) / np.sqrt(d)).astype(np.float32)
        code = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16}[kind]
        self.layer = qs.MoeLayer(code, to_dev(self.router), *dev, f, k, *scales)

    def reference(self, t):
        """moe.layer's dst and bound, every expert on every token (top_k = E)."""
        import torch
        x = self.x[:t].astype(np.float64)
        ids, w = moe.select(x, self.router, 2, True)
        c = ACT_EPS + sum_eps(max(LONG["d"], LONG["f"]))
        xd, ex = to_dev(x), to_dev(c * np.abs(x) + moe.act_error(x))
        dst, err = torch.zeros_like(xd), torch.zeros_like(xd)
        for e in range(LONG["e"]):
            gate, up, down = (v[e] for v in self.values)
            p = to_dev(np.sum(np.where(ids == e, w, 0), axis=1))[:, None]
            g, u = xd @ gate.t(), xd @ up.t()
            eg, eu = ex @ gate.abs().t(), ex @ up.abs().t()
            s = g / (1 + torch.exp(-g))
            h = s * u
            eh = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * h.abs()
            y = h @ down.t()
            held = to_dev(moe.act_error(to_host(h.abs() + eh))) + c * (h.abs() + eh)
            dst += p * y
            err += p * ((eh + held) @ down.abs().t() + 2.0 ** -20 * y.abs())
        return to_host(dst), ids, w, to_host(err)


@pytest.mark.parametrize("kind", KINDS)
def test_waves_take_several_units_of_several_row_groups(kind):
    """3 to 100 tokens on both experts: passes of up to 4, 8 and 16, down in several slices of 64- and 32-row workgroups and
    in one of 16-row ones; repeated calls give the same bits."""
    import torch
    say("moe long", kind)
    qs = _qs()
    m = LongLayer(kind)
    for t in LONG_PLANS:
        say("moe long", kind, t)
        x = to_dev(m.x[:t])
        got = qs.moe_f32(m.layer, x)
        dst, ids, w = (to_host(v) for v in got)
        rd, ri, rw, err = m.reference(t)
        assert np.array_equal(ids, ri) and np.all(np.abs(w - rw) <= 2.0 ** -20 * rw), t
        assert np.all(np.abs(dst - rd) <= err), f"{t}: {np.max(np.abs(dst - rd) / err):.3g} of the bound"
        assert np.linalg.norm(dst - rd) <= 3e-6 * np.linalg.norm(rd), t
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(got, qs.moe_f32(m.layer, x))), t


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,e,top_k", [(1, 300, 4), (2, 200, 16), (4, 512, 1)])
def test_few_tokens_with_the_selection_launched_by_itself(kind, t, e, top_k):
    say("moe select", kind, t, e, top_k)
    m = Layer(kind, t, 96, 64, e, top_k, t + e)
    m.check(_qs().moe_f32(m.layer, to_dev(m.x)), what=f"{kind} T={t} E={e} k={top_k}")


@pytest.mark.parametrize("kind", KINDS)
def test_many_tokens_with_down_in_slices_of_16_rows(kind):
    say("moe slices", kind)
    qs = _qs()
    m = Layer(kind, 70, 96, 16416, 2, 2, 29)
    got = qs.moe_f32(m.layer, to_dev(m.x))
    m.check(got, what=kind)
    assert all(np.array_equal(to_host(a), to_host(b)) for a, b in zip(got, qs.moe_f32(m.layer, to_dev(m.x))))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,e", [(1, 8), (20, 8), (40, 64)])
def test_ids_and_weights_may_be_null(kind, t, e):
    """The C entry point without the two outputs, whoever makes the selection: the same dst."""
    import torch
    say("moe null outputs", kind, t, e)
    qs = _qs()
    m = Layer(kind, t, 96, 64, e, 3, 53)
    x = to_dev(m.x)
    want = qs.moe_f32(m.layer, x)[0]
    ws = torch.full((m.layer.workspace_size(t),), 0xff, dtype=torch.uint8, device="cuda")
    for ids, w in ((None, None), (torch.empty((t, 3), dtype=torch.int32, device="cuda"), None),
                   (None, torch.empty((t, 3), device="cuda"))):
        out = torch.full((t, 96), 7.0, device="cuda")
        st = qs.lib.mm_moe_f32(m.layer._ref, x.data_ptr(), out.data_ptr(), None if ids is None else ids.data_ptr(),
                               None if w is None else w.data_ptr(), t, ws.data_ptr(), ws.numel(),
                               torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(out, want)
