"""Work cases of the 8-bit floating-point product, its quantizer and the mixture-of-experts layer.

Three operators, each in its plain form (elementary torch operations, fp32, fp64 for the router's
logits, whose order decides which experts are taken) and, with ``own`` true, as calls of the library:

* ``quant``: float32 -> e4m3 codes with one float32 scale per 1 x 128 (activations) or 128 x 128
  (weights) block: d = max(amax / 448, 2^-126), code = e4m3(x * (1 / d)), round to nearest even.
* ``mm``: dst[M, N] = a[M, K] . w[N, K]^T, w in e4m3 with 128 x 128 scales, a quantized per 1 x 128
  block within the call (``given`` false) or handed over quantized (``given`` true).
* ``moe``: logits = x . router^T, softmax, the top_k experts of each token (ties: lowest index), their
  probabilities divided by their sum, dst = sum of p_e * down_e(silu(gate_e x) * (up_e x)); experts in
  repacked Q4_0, e4m3 with 128 x 128 scales, or float16.
"""
import math

import torch

own = False

B = 128


def listed():
    return [
        # activations of a prefill step ahead of several products
        {"name": "quant act 512x4096", "op": "quant", "rows": 512, "k": 4096, "block_rows": 1},
        # weights of one projection at load time
        {"name": "quant weight 11008x4096", "op": "quant", "rows": 11008, "k": 4096, "block_rows": 128},
        # one sequence's decode step: attention projection (smallest, latency counts)
        {"name": "mm 1x4096x4096", "op": "mm", "m": 1, "n": 4096, "k": 4096, "given": False},
        # a few sequences, ragged blocks on both axes
        {"name": "mm 5x1000x4128", "op": "mm", "m": 5, "n": 1000, "k": 4128, "given": False},
        # batched decode: ffn up
        {"name": "mm 16x14336x4096", "op": "mm", "m": 16, "n": 14336, "k": 4096, "given": False},
        # larger batch: ffn down, activations quantized by the producer
        {"name": "mm 128x4096x14336", "op": "mm", "m": 128, "n": 4096, "k": 14336, "given": True},
        # prefill: ffn up
        {"name": "mm 512x14336x4096", "op": "mm", "m": 512, "n": 14336, "k": 4096, "given": False},
        # prefill: output projection (largest)
        {"name": "mm 512x128256x4096", "op": "mm", "m": 512, "n": 128256, "k": 4096, "given": True},
        # one token through many small experts (latency counts)
        {"name": "moe q4 T1 E64", "op": "moe", "type": "q4_0r", "t": 1, "d": 2048, "f": 1024, "e": 64, "top_k": 8},
        # a few tokens, sizes that end inside a block, experts in e4m3
        {"name": "moe f8 T7 E12", "op": "moe", "type": "f8", "t": 7, "d": 2080, "f": 1056, "e": 12, "top_k": 3},
        # sixteen sequences, float16 experts
        {"name": "moe f16 T16 E8", "op": "moe", "type": "f16", "t": 16, "d": 2048, "f": 5632, "e": 8, "top_k": 2},
        # a batch through a few large experts
        {"name": "moe q4 T32 E8", "op": "moe", "type": "q4_0r", "t": 32, "d": 4096, "f": 14336, "e": 8, "top_k": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "mm", "mm", "mm", "moe", "moe"))
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 12000), "k": 32 * _log(rng, 1, 448), "block_rows": rng.choice((1, 128))}
    if op == "mm":
        return {"op": op, "m": _log(rng, 1, 512), "n": _log(rng, 16, 20000), "k": 32 * _log(rng, 4, 448),
                "given": rng.random() < 0.3}
    e = rng.randint(2, 64)
    d, f = 32 * _log(rng, 8, 128), 32 * _log(rng, 8, 256)
    f = max(32, min(f, 32 * int(2.0e8 / (e * d * 32))))
    return {"op": op, "type": rng.choice(("q4_0r", "f8", "f16")), "t": _log(rng, 1, 64), "d": d, "f": f, "e": e,
            "top_k": rng.randint(1, min(e, 8))}


def _up(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _act(g, rows, k):
    # a hidden state: unit scale, a few large channels
    return _randn(g, rows, k) * (1 + 7 * (_rand(g, 1, k) < 0.01))


def _f8_weights(g, *shape):
    codes = (_randn(g, *shape) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scale = 2e-4 * (0.75 + 0.5 * _rand(g, *shape[:-2], _up(shape[-2], B), _up(shape[-1], B)))
    return codes, scale


def _q4_0r_weights(g, e, n, k):
    """Repacked Q4_0 experts, [E, ceil(N/16) * ceil(K/256) * 2304] bytes: per tile of 16 rows and
    phase of 8 blocks of 32, 2048 bytes of codes [half][lane][4 blocks][4 bytes] (lane = row + 16 g:
    bytes 4g..4g+3 of that row's block) and the fp16 scales [row][block]."""
    tiles, phases = _up(n, 16), _up(k, 256)
    # byte j of a lane's dword: low nibble element 4g + j of the block, high nibble element 16 + 4g + j
    q = torch.empty(e, tiles, phases, 2048, 2, device="cuda")
    q.normal_(generator=g).mul_(2.5).add_(8.0).round_().clamp_(0, 15)
    codes = (q[..., 0] + 16 * q[..., 1]).to(torch.uint8)
    scale = (0.008 * (0.75 + 0.5 * _rand(g, e, tiles, phases, 16, 8))).half()
    # blocks past K: code 8, scale 0
    blocks = torch.arange(phases * 8, device="cuda").view(phases, 8) >= k // 32
    scale.masked_fill_(blocks[None, None, :, None, :], 0.0)
    pad = blocks.view(1, 1, phases, 2, 1, 4, 1).expand(e, tiles, phases, 2, 64, 4, 4).reshape(e, tiles, phases, 2048)
    codes.masked_fill_(pad, 0x88)
    return torch.cat((codes, scale.view(torch.uint8).reshape(e, tiles, phases, 256)), dim=-1).reshape(e, -1)


def _experts(g, kind, e, n, k):
    if kind == "q4_0r":
        return _q4_0r_weights(g, e, n, k), None
    if kind == "f8":
        return _f8_weights(g, e, n, k)
    return (_randn(g, e, n, k) * 0.02).half(), None


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quant":
        s["x"] = _act(g, case["rows"], case["k"]) * (1.0 if case["block_rows"] == 1 else 0.02)
    elif case["op"] == "mm":
        s["w"], s["w_scale"] = _f8_weights(g, case["n"], case["k"])
        s["x"] = _act(g, case["m"], case["k"])
        if case["given"]:
            s["a"], s["a_scale"] = _quantize(s.pop("x"), 1)
        s["out"] = torch.empty(case["m"], case["n"], device="cuda")
    else:
        t, d, f, e = case["t"], case["d"], case["f"], case["e"]
        s["x"] = _act(g, t, d)
        s["router"] = _randn(g, e, d) / math.sqrt(d)
        for name, n, k in (("gate", f, d), ("up", f, d), ("down", d, f)):
            s[name], s[name + "_scale"] = _experts(g, case["type"], e, n, k)
        s["out"] = torch.empty(t, d, device="cuda")
    return s


# ---------------------------------------------------------------- plain form

def _spread(scale, rows, n, k):
    """Block scales [..., ceil(n/rows), ceil(k/128)] as one value per element."""
    return scale.repeat_interleave(rows, -2)[..., :n, :].repeat_interleave(B, -1)[..., :k]


def _quantize(x, block_rows):
    n, k = x.shape
    rb, kb = _up(n, block_rows), _up(k, B)
    p = torch.zeros(rb * block_rows, kb * B, device=x.device)
    p[:n, :k] = x
    amax = p.view(rb, block_rows, kb, B).abs().amax(dim=(1, 3))
    # both quotients correctly rounded to float32 (by way of float64): a code next to a border depends on them
    d = (amax.double() / 448).float().clamp_min(2.0 ** -126)
    inv = (1 / d.double()).float()
    return (x * _spread(inv, block_rows, n, k)).to(torch.float8_e4m3fn), d


def _f8_values(codes, scale):
    n, k = codes.shape[-2:]
    return codes.float() * _spread(scale, B, n, k)


def _q4_0r_values(w, n, k):
    e, tiles, phases = w.shape[0], _up(n, 16), _up(k, 256)
    w = w.view(e, tiles, phases, 2304)
    c = w[..., :2048].reshape(e, tiles, phases, 2, 4, 16, 4, 4)   # [half][g][row][block][byte]
    c = torch.stack((c & 15, c >> 4), dim=-3).float() - 8.0       # [half][g][row][nibble][block][byte]
    d = w[..., 2048:].contiguous().view(torch.float16).float().view(e, tiles, phases, 16, 2, 4)
    # element of a block: 16 nibble + 4 g + byte
    v = c.permute(0, 1, 5, 2, 3, 7, 6, 4, 8) * d.permute(0, 1, 3, 2, 4, 5)[..., None, None, None]
    return v.reshape(e, tiles * 16, phases * 256)[:, :n, :k]


def _values(s, name, which, n, k):
    """The chosen experts' weights as float32, [len(which), n, k]."""
    w = s[name][which] if s["type"] != "f8" else s[name].view(torch.uint8)[which].view(torch.float8_e4m3fn)
    if s["type"] == "q4_0r":
        return _q4_0r_values(w, n, k)
    if s["type"] == "f8":
        return _f8_values(w, s[name + "_scale"][which])
    return w.float()


def _moe(s):
    x, d, f, e, k = s["x"], s["d"], s["f"], s["e"], s["top_k"]
    t = x.shape[0]
    p = torch.softmax(x.double() @ s["router"].double().t(), dim=-1)
    p, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]
    p = (p / p.sum(dim=-1, keepdim=True)).float()
    if t * k <= e:   # few: the chosen experts' weights, one copy per use
        which, rows = ids.reshape(-1), x.repeat_interleave(k, 0)[:, None, :]
        mix = p.reshape(t, 1, k)
    else:            # many: every expert on every token
        which, rows = torch.arange(e, device=x.device), x[None].expand(e, t, d)
        mix = torch.zeros(t, e, device=x.device).scatter_(1, ids, p).t()[:, :, None]
    gate = torch.bmm(rows, _values(s, "gate", which, f, d).transpose(1, 2).contiguous())
    up = torch.bmm(rows, _values(s, "up", which, f, d).transpose(1, 2).contiguous())
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(h, _values(s, "down", which, d, f).transpose(1, 2).contiguous())
    y = torch.bmm(mix, y.view(t, k, d))[:, 0] if t * k <= e else (mix * y).sum(0)
    return {"dst": y, "ids": ids.to(torch.int32), "weights": p}


def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "quant":
        return _quantize(s["x"], s["block_rows"])
    if s["op"] == "mm":
        a, a_scale = (s["a"], s["a_scale"]) if s["given"] else _quantize(s["x"], 1)
        a = a.float() * _spread(a_scale, 1, s["m"], s["k"])
        return a @ _f8_values(s["w"], s["w_scale"]).t()
    return _moe(s)


def _own(s):
    import quantized_skinny_gemm_amd as qs
    if s["op"] == "quant":
        return qs.quantize_f8(s["x"], s["block_rows"])
    if s["op"] == "mm":
        if "ws" not in s:
            s["ws"] = torch.empty(qs.f8_workspace_size(s["m"], s["n"], s["k"], s["given"]), dtype=torch.uint8, device="cuda")
        if s["given"]:
            return qs.mul_mat_f8_f8(s["w"], s["w_scale"], s["a"], s["a_scale"], out=s["out"], ws=s["ws"])
        return qs.mul_mat_f8_f32(s["w"], s["w_scale"], s["x"], out=s["out"], ws=s["ws"])
    if "layer" not in s:
        kind = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16}[s["type"]]
        s["layer"] = qs.MoeLayer(kind, s["router"], s["gate"], s["up"], s["down"], s["f"], s["top_k"],
                                 s["gate_scale"], s["up_scale"], s["down_scale"])
        s["ws"] = torch.empty(s["layer"].workspace_size(s["t"]), dtype=torch.uint8, device="cuda")
    dst, ids, weights = qs.moe_f32(s["layer"], s["x"], out=s["out"], ws=s["ws"])
    return {"dst": dst, "ids": ids, "weights": weights}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "quant":
        n, k, r = case["rows"], case["k"], case["block_rows"]
        return {"bytes": 5 * n * k + 4 * _up(n, r) * _up(k, B), "flops": 3 * n * k}
    if case["op"] == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        act = m * k + 4 * m * _up(k, B) if case["given"] else 4 * m * k
        return {"bytes": n * k + 4 * _up(n, B) * _up(k, B) + act + 4 * m * n, "flops": 2 * m * n * k}
    t, d, f, e, k = (case[x] for x in ("t", "d", "f", "e", "top_k"))
    used = e * (1 - (1 - k / e) ** t)          # experts that at least one token takes, on average
    per = {"q4_0r": 18 / 32, "f8": 1 + 4 / (B * B), "f16": 2}[case["type"]]
    return {"bytes": used * 3 * d * f * per + 4 * e * d + 8 * t * d, "flops": 2 * t * e * d + 6 * t * k * d * f}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_e4m3(v):
    """float64 -> nearest e4m3 value (ties to even): 3 fraction bits, exponents from -6, largest 448."""
    e = torch.frexp(v.abs())[1] - 1                     # 2^e <= |v| < 2^(e+1)
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_bits(codes):
    """Value of an e4m3 byte: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    b = codes.view(torch.uint8).to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, -9)), torch.ldexp(8 + m, e - 10))
    return torch.where(b >= 128, -v, v)


def _exact_quant(x, r):
    """Codes' values and scales; the definition fixes each step as one float32 rounding, taken here from float64
    results that hold the exact (or innocuously rounded) quotient or product."""
    n, k = x.shape
    ri = (torch.arange(n, device=x.device) // r)[:, None]
    ki = (torch.arange(k, device=x.device) // B)[None, :]
    nb, kb = _up(n, r), _up(k, B)
    block = (ri * kb + ki).reshape(-1)
    amax = torch.zeros(nb * kb, dtype=torch.float64, device=x.device)
    amax.scatter_reduce_(0, block, x.double().abs().reshape(-1), "amax")
    d = (amax / 448).float().clamp_min(2.0 ** -126)
    inv = (1 / d.double()).float()
    v = (x.double() * inv.double()[block].view(n, k)).float()
    return _exact_e4m3(v.double()), d.view(nb, kb)


def _exact_experts(s, name, e, n, k):
    w = s[name][e]
    if s["type"] == "f16":
        return w.double()
    if s["type"] == "f8":
        i = torch.arange(n, device="cuda")[:, None] // B
        j = torch.arange(k, device="cuda")[None, :] // B
        return _exact_bits(w) * s[name + "_scale"][e].double()[i, j]
    # Q4_0R, one gather per byte: where row i, element c of a row of k values lies
    i = torch.arange(n, device="cuda")[:, None]
    c = torch.arange(k, device="cuda")[None, :]
    chunk = ((i // 16) * _up(k, 256) + c // 256) * 2304
    blk, el = (c % 256) // 32, c % 32
    lane = i % 16 + 16 * ((el % 16) // 4)
    byte = w[chunk + (blk // 4) * 1024 + lane * 16 + (blk % 4) * 4 + el % 4].to(torch.int32)
    code = torch.where(el >= 16, byte >> 4, byte & 15) - 8
    at = chunk + 2048 + (i % 16) * 16 + blk * 2
    half = (w[at].to(torch.int32) + 256 * w[at + 1].to(torch.int32)).to(torch.int16).view(torch.float16)
    return code.double() * half.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        codes, d = _exact_quant(s["x"], case["block_rows"])
        return codes, d.double()
    if case["op"] == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        codes, d = (_exact_bits(s["a"]), s["a_scale"]) if case["given"] else _exact_quant(s["x"], 1)
        kb = torch.arange(k, device="cuda") // B
        a = codes * d.double()[:, kb]
        dst = torch.empty(m, n, dtype=torch.float64, device="cuda")
        for r in range(0, n, 8192):
            rows = torch.arange(r, min(r + 8192, n), device="cuda")
            w = _exact_bits(s["w"][r:r + 8192]) * s["w_scale"].double()[rows // B][:, kb]
            dst[:, rows] = a @ w.t()
        return dst
    x, t, k = s["x"].double(), case["t"], case["top_k"]
    logits = x @ s["router"].double().t()
    z = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    p = z / z.sum(dim=1, keepdim=True)
    dst = torch.zeros(t, case["d"], dtype=torch.float64, device="cuda")
    ids = torch.empty(t, k, dtype=torch.int32, device="cuda")
    left, chosen = p.clone(), torch.empty(t, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        chosen[:, j], at = left.max(dim=1)
        ids[:, j] = at.to(torch.int32)
        left[torch.arange(t, device="cuda"), at] = -1
    weights = chosen / chosen.sum(dim=1, keepdim=True)
    for e in range(case["e"]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if len(tok):
            g = x[tok] @ _exact_experts(s, "gate", e, case["f"], case["d"]).t()
            u = x[tok] @ _exact_experts(s, "up", e, case["f"], case["d"]).t()
            y = (g / (1 + torch.exp(-g)) * u) @ _exact_experts(s, "down", e, case["d"], case["f"]).t()
            dst[tok] += weights[tok, slot][:, None] * y
    return {"dst": dst, "ids": ids, "weights": weights}
