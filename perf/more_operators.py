"""Work cases of the microscaled 4-bit product and its quantizer, the root-mean-square norm, the routing to experts and
the experts' products for a given routing.

Five operators, each in its plain form (elementary torch operations in fp32; fp64 for the norm's mean and the routing's
scores, which decide codes and choices next to a border) and, with ``own`` true, as calls of the library:

* ``quant``: float32 -> MXFP4 and back: 32 values along K share a scale 2^e, e = max(floor(log2(amax)) - 2, -127); code =
  e2m1(x / 2^e) (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), ties to the even code, larger magnitudes give 6.
* ``mm``: dst[M, N] = a[M, K] . w[N, K]^T, both in MXFP4; a quantized within the call (``given`` false) or handed over so.
* ``norm``: v = x + residual, y = (v * rstd) * weight, rstd = 1 / sqrt(mean(v^2) + eps); v, and y in float32, as e4m3 codes
  with a float32 scale per 128 values (d = max(amax / 448, 2^-126), code = e4m3(y * (1 / d))), or as MXFP4.
* ``route``: scores s = softmax or sigmoid of the logits; chosen by s + bias within the best groups (a group's value: the
  sum of its two best), ties to the lower index; weights: the chosen s over their sum, times a factor.
* ``experts``: dst = sum over a token's experts of weight * down(silu(gate x) * (up x)), experts in MXFP4, x as it is.
"""
import math

import torch

own = False

B = 32
EPS = 1e-5


def listed():
    return [
        # activations of a prefill step, there and back: what a user looks at to judge the format
        {"name": "quant act 511x4096", "op": "quant", "rows": 511, "k": 4096, "std": 1.0},
        # weights of one projection at load time
        {"name": "quant weight 11008x4096", "op": "quant", "rows": 11008, "k": 4096, "std": 0.02},
        # one sequence's decode step: attention projection (latency counts)
        {"name": "mm 1x4096x4096", "op": "mm", "m": 1, "n": 4096, "k": 4096, "given": False},
        # a few sequences, sizes that end inside every tile
        {"name": "mm 7x1000x4128", "op": "mm", "m": 7, "n": 1000, "k": 4128, "given": False},
        # batched decode: ffn up, activations quantized by the norm ahead of it
        {"name": "mm 32x14336x4096", "op": "mm", "m": 32, "n": 14336, "k": 4096, "given": True},
        # prefill: output projection (largest)
        {"name": "mm 512x128256x4096", "op": "mm", "m": 512, "n": 128256, "k": 4096, "given": False},
        # one token ahead of the attention projections (smallest)
        {"name": "norm f8 1x4096", "op": "norm", "t": 1, "d": 4096, "out": "f8"},
        # a prefill step ahead of the ffn
        {"name": "norm mxfp4 2047x8192", "op": "norm", "t": 2047, "d": 8192, "out": "mxfp4"},
        # one token, many experts in groups
        {"name": "route sigmoid T1 E256", "op": "route", "t": 1, "e": 256, "top_k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "group_k": 4, "norm": True, "scale": 2.5},
        # a prefill step
        {"name": "route softmax T4095 E64", "op": "route", "t": 4095, "e": 64, "top_k": 6, "score": "softmax", "bias": False,
         "groups": 1, "group_k": 1, "norm": True, "scale": 1.0},
        # one token through a few of many small experts
        {"name": "experts T1 E64", "op": "experts", "t": 1, "d": 2048, "f": 1024, "e": 64, "top_k": 8},
        # a batch through large experts
        {"name": "experts T32 E8", "op": "experts", "t": 32, "d": 4096, "f": 14336, "e": 8, "top_k": 2},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "mm", "mm", "mm", "norm", "norm", "route", "route", "experts", "experts"))
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 12000), "k": B * _log(rng, 1, 448), "std": rng.choice((1.0, 0.02))}
    if op == "mm":
        return {"op": op, "m": _log(rng, 1, 512), "n": _log(rng, 16, 20000), "k": B * _log(rng, 4, 448),
                "given": rng.random() < 0.4}
    if op == "norm":
        out = rng.choice(("f32", "f8", "mxfp4"))
        return {"op": op, "t": _log(rng, 1, 4096), "d": _log(rng, 16, 16384) if out == "f32" else B * _log(rng, 2, 512),
                "out": out}
    if op == "route":
        groups, per = rng.choice((1, 1, 4, 8)), rng.randint(4, 64)
        group_k = rng.randint(1, groups)
        return {"op": op, "t": _log(rng, 1, 8192), "e": groups * per, "top_k": rng.randint(1, min(8, group_k * per)),
                "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups,
                "group_k": group_k, "norm": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5))}
    e = rng.randint(2, 64)
    d, f = B * _log(rng, 8, 128), B * _log(rng, 8, 256)
    f = max(B, min(f, B * int(2.0e8 / (e * d * B))))
    return {"op": op, "t": _log(rng, 1, 64), "d": d, "f": f, "e": e, "top_k": rng.randint(1, min(e, 8))}


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


def _scale_bytes(e, k):
    """Scale exponents [..., K/32] as bytes, rows padded with 127 to whole 4 bytes."""
    s = torch.full((*e.shape[:-1], 4 * _up(k, 4 * B)), 127, dtype=torch.uint8, device=e.device)
    s[..., :k // B] = (e + 127).to(torch.uint8)
    return s


def _weights(g, *shape):
    """MXFP4 weights of about 0.02: codes as a normal distribution gives them, scales around 2^-7; bytes [..., N, K/2]
    (element 2 i in the low half of byte i) and scale bytes."""
    q = 2.7 * torch.special.ndtri((torch.arange(64, device="cuda") + 0.5) / 64)
    nib = _codes(q)
    pairs = (nib[None, :] + 16 * nib[:, None]).reshape(-1).to(torch.uint8)
    k = shape[-1]
    at = torch.randint(0, 4096, (*shape[:-1], k // 2), generator=g, device="cuda", dtype=torch.int32)
    e = torch.randint(-8, -5, (*shape[:-1], k // B), generator=g, device="cuda", dtype=torch.int32)
    return pairs[at], _scale_bytes(e, k)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "quant":
        s["x"] = _act(g, case["rows"], case["k"]) * case["std"]
    elif op == "mm":
        s["w"], s["w_scale"] = _weights(g, case["n"], case["k"])
        x = _act(g, case["m"], case["k"])
        if case["given"]:
            values, e = _quantize(x)
            codes = _codes(torch.ldexp(values, -e.repeat_interleave(B, -1)))
            s["a"] = (codes[:, 0::2] + 16 * codes[:, 1::2]).to(torch.uint8)
            s["a_scale"] = _scale_bytes(e, case["k"])
        else:
            s["x"] = x
        s["out"] = torch.empty(case["m"], case["n"], device="cuda")
    elif op == "norm":
        s["x"] = _act(g, case["t"], case["d"])
        s["residual"] = 4 * _act(g, case["t"], case["d"])
        s["weight"] = 1 + 0.2 * _randn(g, case["d"])
    elif op == "route":
        s["logits"] = 1.5 * _randn(g, case["t"], case["e"])
        s["b"] = 0.05 * _randn(g, case["e"]) if case["bias"] else None
    else:
        t, d, f, e, k = (case[n] for n in ("t", "d", "f", "e", "top_k"))
        s["x"] = _act(g, t, d)
        for name, n, m in (("gate", f, d), ("up", f, d), ("down", d, f)):
            s[name], s[name + "_scale"] = _weights(g, e, n, m)
        s["ids"] = torch.argsort(_rand(g, t, e), dim=-1)[:, :k].to(torch.int32).contiguous()
        w = 0.2 + _rand(g, t, k)
        s["weights"] = w / w.sum(dim=-1, keepdim=True)
        s["out"] = torch.empty(t, d, device="cuda")
    return s


# ---------------------------------------------------------------- plain form

def _codes(v):
    """Code (sign in bit 3) of the e2m1 value nearest to v, ties to the even code."""
    a = v.abs()
    c = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return c + 8 * (v < 0).int()


def _quantize(x):
    """(values float32 [rows, K], scale exponents int32 [rows, K/32]) of x in MXFP4."""
    n, k = x.shape
    amax = x.view(n, k // B, B).abs().amax(dim=2)
    e = (torch.frexp(amax)[1] - 3).clamp_min(-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    spread = e.repeat_interleave(B, 1)
    a = torch.ldexp(x, -spread).abs()
    v = (0.5 * ((a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float())
         + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5.0).float())
    return torch.ldexp(torch.where(x < 0, -v, v), spread), e


def _values(codes, scale, k):
    """float32 values [..., K] of packed codes and scale bytes."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    e = torch.exp2(scale[..., :k // B].float() - 127)
    return table[c.int()] * e.repeat_interleave(B, -1)


def _norm(s):
    v = s["x"] + s["residual"]
    d = v.double()
    eps = float(torch.tensor(EPS, dtype=torch.float32))
    rstd = (1 / torch.sqrt(d.square().mean(dim=1, keepdim=True) + eps)).float()
    y = (v * rstd) * s["weight"]
    if s["out"] == "f32":
        return {"y": y, "sum": v}
    if s["out"] == "mxfp4":
        return {"values": _quantize(y)[0], "sum": v}
    t, n = y.shape
    kb = _up(n, 128)
    p = torch.zeros(t, kb * 128, device=y.device)
    p[:, :n] = y
    amax = p.view(t, kb, 128).abs().amax(dim=2)
    scales = (amax.double() / 448).float().clamp_min(2.0 ** -126)
    inv = (1 / scales.double()).float()
    codes = (y * inv.repeat_interleave(128, 1)[:, :n]).to(torch.float8_e4m3fn)
    return {"codes": codes, "scales": scales, "sum": v}


def _route(s):
    l = s["logits"].double()
    t, e = l.shape
    if s["score"] == "softmax":
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    c = p if s["b"] is None else p + s["b"].double()
    if s["groups"] > 1:
        g = c.view(t, s["groups"], e // s["groups"])
        two = torch.sort(g, dim=2, descending=True)[0][:, :, :2].sum(dim=2)
        best = torch.sort(two, dim=1, descending=True, stable=True)[1][:, :s["group_k"]]
        keep = torch.zeros(t, s["groups"], dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = torch.where(keep[:, :, None], g, torch.full_like(g, -math.inf)).view(t, e)
    ids = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :s["top_k"]]
    w = torch.gather(p, 1, ids)
    if s["norm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * s["scale"]).float()}


def _experts(s):
    x, d, f, e, k = s["x"], s["d"], s["f"], s["e"], s["top_k"]
    t = x.shape[0]
    ids = s["ids"].long()
    if t * k <= e:   # few: the chosen experts' weights, one copy per use
        which, rows = ids.reshape(-1), x.repeat_interleave(k, 0)[:, None, :]
    else:            # many: every expert on every token
        which, rows = torch.arange(e, device=x.device), x[None].expand(e, t, d)
    gate = torch.bmm(rows, _values(s["gate"][which], s["gate_scale"][which], d).transpose(1, 2).contiguous())
    up = torch.bmm(rows, _values(s["up"][which], s["up_scale"][which], d).transpose(1, 2).contiguous())
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(h, _values(s["down"][which], s["down_scale"][which], f).transpose(1, 2).contiguous())
    if t * k <= e:
        return (s["weights"][:, :, None] * y.view(t, k, d)).sum(dim=1)
    mix = torch.zeros(t, e, device=x.device).scatter_(1, ids, s["weights"])
    return (mix.t()[:, :, None] * y).sum(dim=0)


def run(state):
    s = state
    if own:
        return _own(s)
    op = s["op"]
    if op == "quant":
        return {"values": _quantize(s["x"])[0]}
    if op == "mm":
        a = _values(s["a"], s["a_scale"], s["k"]) if s["given"] else _quantize(s["x"])[0]
        return a @ _values(s["w"], s["w_scale"], s["k"]).t()
    if op == "norm":
        return _norm(s)
    if op == "route":
        return _route(s)
    return _experts(s)


def _own(s):
    import quantized_skinny_gemm_amd as qs
    op = s["op"]
    if op == "quant":
        codes, scales = qs.quantize_mxfp4(s["x"])
        return {"values": qs.dequantize_mxfp4(codes, scales)}
    if op == "mm":
        if "ws" not in s:
            s["ws"] = torch.empty(qs.mxfp4_workspace_size(s["m"], s["n"], s["k"], s["given"]), dtype=torch.uint8, device="cuda")
        if s["given"]:
            return qs.mul_mat_mxfp4_mxfp4(s["w"], s["w_scale"], s["a"], s["a_scale"], out=s["out"], ws=s["ws"])
        return qs.mul_mat_mxfp4_f32(s["w"], s["w_scale"], s["x"], out=s["out"], ws=s["ws"])
    if op == "norm":
        kind = {"f32": qs.MM_TYPE_F32, "f8": qs.MM_TYPE_F8, "mxfp4": qs.MM_TYPE_MXFP4}[s["out"]]
        y, v = qs.rms_norm_f32(s["x"], s["weight"], EPS, residual=s["residual"], out_type=kind)
        if s["out"] == "f32":
            return {"y": y, "sum": v}
        if s["out"] == "f8":
            return {"codes": y[0], "scales": y[1], "sum": v}
        return {"values": qs.dequantize_mxfp4(*y), "sum": v}
    if op == "route":
        if "router" not in s:
            s["router"] = qs.Router(s["e"], s["top_k"], score=s["score"], bias=s["b"], groups=s["groups"],
                                    group_k=s["group_k"], group_top=2 if s["groups"] > 1 else 1, norm=s["norm"], scale=s["scale"])
        ids, weights = qs.route_f32(s["router"], s["logits"])
        return {"ids": ids, "weights": weights}
    if "layer" not in s:
        s["layer"] = qs.MoeLayer(qs.MM_TYPE_MXFP4, None, s["gate"], s["up"], s["down"], s["f"], s["top_k"],
                                 s["gate_scale"], s["up_scale"], s["down_scale"])
        s["ws"] = torch.empty(s["layer"].routed_workspace_size(s["t"]), dtype=torch.uint8, device="cuda")
    return qs.moe_routed_f32(s["layer"], s["x"], s["ids"], s["weights"], out=s["out"], ws=s["ws"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["k"]            # values to codes and scales, and those to values
        return {"bytes": 2 * (4 + 17 / 32) * n, "flops": 4 * n}
    if op == "mm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 17 / 32 * n * k + (17 / 32 if case["given"] else 4) * m * k + 4 * m * n, "flops": 2 * m * n * k}
    if op == "norm":
        # x, residual, v; y, through its codes for values
        n, per = case["t"] * case["d"], {"f32": 4, "f8": 1 + 4 / 128, "mxfp4": 2 * 17 / 32 + 4}[case["out"]]
        return {"bytes": (12 + per) * n + 4 * case["d"], "flops": 6 * n}
    if op == "route":
        return {"bytes": 4 * case["t"] * case["e"] + 8 * case["t"] * case["top_k"], "flops": 8 * case["t"] * case["e"]}
    t, d, f, e, k = (case[x] for x in ("t", "d", "f", "e", "top_k"))
    used = e * (1 - (1 - k / e) ** t)          # experts that at least one token takes, on average
    return {"bytes": used * 3 * d * f * 17 / 32 + 8 * t * d + 8 * t * k, "flops": 6 * t * k * d * f}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_e2m1(v):
    """float64 -> nearest e2m1 value (ties to even): 1 fraction bit, exponents from 0, largest 6."""
    e = (torch.frexp(v.abs())[1] - 1).clamp_min(0)
    step = torch.ldexp(torch.ones_like(v), e - 1)
    return (torch.round(v / step) * step).clamp(-6, 6)


def _exact_quant(x):
    """float64 [rows, K] -> the MXFP4 values nearest to it."""
    n, k = x.shape
    block = x.view(n, k // B, B)
    top = block.abs().amax(dim=2, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -125.0))
    # log2 rounds: next to a power of two the exponent is settled by comparison
    e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double() * (top > 0)
    unit = torch.exp2((e - 2).clamp_min(-127))
    return (_exact_e2m1(block / unit) * unit).view(n, k)


def _exact_e4m3(v):
    """float64 -> nearest e4m3 value (ties to even): 3 fraction bits, exponents from -6, largest 448."""
    e = torch.frexp(v.abs())[1] - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_values(codes, scale):
    """Values of packed codes [N, K/2]: sign, 2 exponent bits (bias 1), 1 fraction bit; times 2^(byte - 127)."""
    n, half = codes.shape
    c = torch.empty(n, 2 * half, dtype=torch.int32, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    e, m = (c // 2) % 4, (c % 2).double()
    v = torch.where(e == 0, m / 2, torch.ldexp(1 + m / 2, e - 1))
    at = torch.arange(2 * half, device=codes.device) // B
    return torch.ldexp(torch.where(c >= 8, -v, v), scale[:, at].to(torch.int32) - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        return {"values": _exact_quant(s["x"].double())}
    if op == "mm":
        m, n = case["m"], case["n"]
        a = _exact_values(s["a"], s["a_scale"]) if case["given"] else _exact_quant(s["x"].double())
        dst = torch.empty(m, n, dtype=torch.float64, device="cuda")
        for r in range(0, n, 8192):
            dst[:, r:r + 8192] = a @ _exact_values(s["w"][r:r + 8192], s["w_scale"][r:r + 8192]).t()
        return dst
    if op == "norm":
        # v is a float32 output of its own; y starts from it
        v = (s["x"].double() + s["residual"].double()).float().double()
        n, w = case["d"], s["weight"].double()
        root = ((v * v).sum(dim=1, keepdim=True) / n + torch.tensor(EPS).double().item()).sqrt()
        if case["out"] == "f32":
            return {"y": v * w / root, "sum": v}
        # what is quantized is y as float32: rstd, v * rstd and the product with weight are rounded to it in turn
        y = ((v * (1 / root).float().double()).float().double() * w).float().double()
        if case["out"] == "mxfp4":
            return {"values": _exact_quant(y), "sum": v}
        at = torch.arange(n, device="cuda") // 128
        d = torch.zeros(case["t"], _up(n, 128), dtype=torch.float64, device="cuda")
        d.scatter_reduce_(1, at.expand(case["t"], n).contiguous(), y.abs(), "amax")
        d = d / 448
        return {"codes": _exact_e4m3(y / d[:, at]), "scales": d, "sum": v}
    if op == "route":
        l = s["logits"].double()
        p = torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)
        t, e, g = case["t"], case["e"], case["groups"]
        c = p + (0 if s["b"] is None else s["b"].double())
        rows = torch.arange(t, device="cuda")
        if g > 1:
            a = c.clone().view(t, g, e // g)
            first, at = a.max(dim=2)
            a.scatter_(2, at[:, :, None], -math.inf)
            value = first + a.amax(dim=2)
            allowed = torch.zeros(t, g, dtype=torch.bool, device="cuda")
            for _ in range(case["group_k"]):
                at = value.max(dim=1)[1]
                allowed[rows, at] = True
                value[rows, at] = -math.inf
            c = c.masked_fill(~allowed.repeat_interleave(e // g, 1), -math.inf)
        ids, w = [], []
        for _ in range(case["top_k"]):
            at = c.max(dim=1)[1]
            ids.append(at)
            w.append(p[rows, at])
            c[rows, at] = -math.inf
        w = torch.stack(w, dim=1)
        w = w / w.sum(dim=1, keepdim=True) if case["norm"] else w
        return {"ids": torch.stack(ids, dim=1).to(torch.int32), "weights": w * case["scale"]}
    x = s["x"].double()
    dst = torch.zeros(case["t"], case["d"], dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        tok, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if len(tok):
            g = x[tok] @ _exact_values(s["gate"][e], s["gate_scale"][e]).t()
            u = x[tok] @ _exact_values(s["up"][e], s["up_scale"][e]).t()
            y = (g / (1 + torch.exp(-g)) * u) @ _exact_values(s["down"][e], s["down_scale"][e]).t()
            dst[tok] += s["weights"].double()[tok, slot][:, None] * y
    return dst
