"""Host-side checks of the MXFP4, norm, routing and routed-experts entry points: arguments are refused before any HIP call
(the pointers here are never dereferenced), workspace sizes, the binding's own checks."""
from __future__ import annotations

import ctypes

import pytest

import quantized_skinny_gemm_amd as qs
from tests.test_f8_moe_host import _as_gpu

OK, NULL, SHAPE, ALIGN, WS, ALIAS, ARG = 0, -1, -2, -3, -4, -5, -8
W, WSC, X, XSC, DST, WSP = (0x7f0000000000 + (i << 36) for i in range(6))
G = 1 << 30


def _f32(m=40, n=256, k=512, w=W, wsc=WSC, x=X, dst=DST, ws=WSP, wsb=None):
    wsb = qs.mxfp4_workspace_size(m, n, k) if wsb is None else wsb
    return qs.lib.mm_mul_mat_mxfp4_f32(w, wsc, x, dst, m, n, k, ws, wsb, None)


def _mx(m=40, n=256, k=512, w=W, wsc=WSC, x=X, xsc=XSC, dst=DST, ws=WSP, wsb=None):
    wsb = qs.mxfp4_workspace_size(m, n, k, True) if wsb is None else wsb
    return qs.lib.mm_mul_mat_mxfp4_mxfp4(w, wsc, x, xsc, dst, m, n, k, ws, wsb, None)


def test_type_and_sizes():
    assert qs.MM_TYPE_MXFP4 == 6
    assert qs.row_bytes(qs.MM_TYPE_MXFP4, 4096) == 2048 and qs.row_bytes(qs.MM_TYPE_MXFP4, 48) == -1
    assert qs.workspace_size(qs.MM_TYPE_MXFP4, 100, 300, 512) == qs.mxfp4_workspace_size(100, 300, 512) >= 100 * 272
    assert qs.mxfp4_workspace_size(-1, 4, 32) == 0 and qs.mxfp4_workspace_size(1, 4, 33) == 0
    assert qs.lib.mm_dispatch(qs.MM_TYPE_MXFP4, 1, 64, 64, None) == ARG
    assert qs.lib.mm_debug_mul_mat(qs.MM_TYPE_MXFP4, W, X, DST, None, 1, 64, 64, 0, 0, 0, None, 0, None) == ARG


@pytest.mark.parametrize("call", [_f32, _mx])
def test_product_refusals(call):
    for bad in (dict(k=48), dict(m=-1), dict(n=-1), dict(k=-32), dict(n=2 ** 31), dict(m=2 ** 31), dict(k=2 ** 23 + 32)):
        assert call(**{**dict(wsb=0), **bad}) == SHAPE, bad
    for p in ("w", "wsc", "x", "dst"):
        assert call(**{p: None}) == NULL, p
    assert call(w=W + 8) == ALIGN and call(wsc=WSC + 2) == ALIGN and call(x=X + 4) == ALIGN and call(dst=DST + 2) == ALIGN
    assert call(dst=W + 4096) == ALIAS and call(dst=X) == ALIAS and call(dst=WSC) == ALIAS
    assert call(m=0, w=None, x=None, dst=None, wsb=0) == OK and call(n=0, w=None, dst=None, wsb=0) == OK
    for m, n, k in ((1, 2 ** 31 - 1, 32), (2 ** 31 - 1, 1, 32), (2 ** 24, 2 ** 17, 32), (2 ** 17, 2 ** 24, 32)):
        assert call(m, n, k, wsb=0) == SHAPE, (m, n, k)


def test_product_workspace_refusals():
    need = qs.mxfp4_workspace_size(40, 256, 512)
    assert need >= 40 * 256 + 40 * 16
    assert _f32(wsb=need - 1) == WS and _f32(ws=None) == WS and _f32(ws=WSP + 64) == ALIGN
    for p in (W, WSC, X, DST):
        assert _f32(ws=p) == ALIAS
    assert _mx(xsc=None) == NULL and _mx(xsc=XSC + 1) == ALIGN and _mx(dst=XSC) == ALIAS


@pytest.mark.parametrize("forward", [True, False])
def test_quantize_refusals(forward):
    def q(x, c, s, rows, k):
        if forward:
            return qs.lib.mm_quantize_mxfp4(x, c, s, rows, k, None)
        return qs.lib.mm_dequantize_mxfp4(c, s, x, rows, k, None)

    assert q(X, W, WSC, 4, 48) == SHAPE and q(X, W, WSC, -1, 64) == SHAPE and q(X, W, WSC, 4, 2 ** 23 + 32) == SHAPE
    for i in range(3):
        p = [X, W, WSC]
        p[i] = None
        assert q(*p, 4, 64) == NULL
    assert q(X + 4, W, WSC, 4, 64) == ALIGN and q(X, W + 8, WSC, 4, 64) == ALIGN and q(X, W, WSC + 2, 4, 64) == ALIGN
    assert q(X, X + 256, WSC, 4, 64) == ALIAS and q(X, W, X + 16, 4, 64) == ALIAS and q(X, W, W, 4, 64) == ALIAS
    assert q(None, None, None, 0, 64) == OK and q(None, None, None, 3, 0) == OK


def _norm(x=X, r=W, g=WSC, eps=1e-5, s=DST, kind=None, y=WSP, sc=XSC, t=4, d=256):
    return qs.lib.mm_rms_norm_f32(x, r, g, eps, s, qs.MM_TYPE_F8 if kind is None else kind, y, sc, t, d, None)


def test_norm_refusals():
    for kind in (qs.MM_TYPE_F16, qs.MM_TYPE_Q4_0, qs.MM_TYPE_Q8_0, 99, -1):
        assert _norm(kind=kind) == ARG
    assert _norm(eps=-1e-6) == ARG and _norm(eps=float("nan")) == ARG
    assert _norm(t=-1) == SHAPE and _norm(d=-1) == SHAPE and _norm(d=48) == SHAPE and _norm(d=2 ** 23 + 32) == SHAPE
    assert _norm(t=2 ** 26, d=32, kind=0) == SHAPE          # 2^32 threads
    assert _norm(t=0, x=None, y=None) == OK and _norm(d=0, x=None, y=None) == OK
    assert _norm(x=None) == NULL and _norm(y=None) == NULL and _norm(sc=None) == NULL
    for kind in (qs.MM_TYPE_F8, qs.MM_TYPE_MXFP4):
        assert _norm(kind=kind, y=WSP + 4) == ALIGN and _norm(kind=kind, sc=XSC + 2) == ALIGN
    assert _norm(x=X + 2) == ALIGN and _norm(r=W + 1) == ALIGN and _norm(g=WSC + 2) == ALIGN and _norm(s=DST + 2) == ALIGN
    assert _norm(kind=0, y=WSP + 2) == ALIGN
    b = 4 * 256 * 4
    for kind in (qs.MM_TYPE_F32, qs.MM_TYPE_F8, qs.MM_TYPE_MXFP4):
        for y in (X, W + b - 16, WSC, DST):
            assert _norm(kind=kind, y=y) == ALIAS, (kind, hex(y))
    assert _norm(s=X + 16) == ALIAS and _norm(s=W - 16) == ALIAS and _norm(s=WSC) == ALIAS
    assert _norm(sc=X) == ALIAS and _norm(sc=WSP) == ALIAS and _norm(sc=DST) == ALIAS


def _router(**kw):
    base = dict(score=0, top_k=2, norm=1, groups=1, group_k=1, group_top=1, E=8, scale=1.0, bias=None)
    base.update(kw)
    return qs._RouterStruct(**base)


def _route(r, l=X, ids=W, w=DST, t=5):
    return qs.lib.mm_route_f32(ctypes.byref(r), l, ids, w, t, None)


def test_route_refusals():
    assert qs.lib.mm_route_f32(None, X, W, DST, 1, None) == NULL
    for bad in (dict(score=2), dict(score=-1), dict(group_top=0), dict(group_top=3)):
        assert _route(_router(**bad)) == ARG, bad
    for bad in (dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=9), dict(top_k=65, E=128), dict(groups=0), dict(groups=3),
                dict(groups=2, group_k=3), dict(groups=2, group_k=0), dict(groups=65, E=130)):
        assert _route(_router(**bad)) == SHAPE, bad
    assert _route(_router(), t=-1) == SHAPE and _route(_router(), t=2 ** 25 + 1) == SHAPE
    assert _route(_router(), t=0, l=None) == OK
    assert _route(_router(), l=None) == NULL and _route(_router(), ids=None) == NULL and _route(_router(), w=None) == NULL
    assert _route(_router(), l=X + 2) == ALIGN and _route(_router(), ids=W + 1) == ALIGN and _route(_router(), w=DST + 2) == ALIGN
    assert _route(_router(bias=WSC + 1)) == ALIGN
    assert _route(_router(), ids=X) == ALIAS and _route(_router(), w=X + 156) == ALIAS and _route(_router(), w=W + 36) == ALIAS
    assert _route(_router(bias=WSC), ids=WSC) == ALIAS and _route(_router(bias=DST)) == ALIAS


def _layer(**kw):
    base = dict(type=qs.MM_TYPE_MXFP4, top_k=2, norm=1, D=256, F=128, E=4, router=None, gate=W, up=W + G, down=W + 2 * G,
                gate_scale=WSC, up_scale=WSC + G, down_scale=WSC + 2 * G)
    base.update(kw)
    return qs._MoeStruct(**base)


def _moe(layer, t=3, x=X, dst=DST, ids=XSC, w=XSC + G, ws=WSP, wsb=None):
    wsb = qs.lib.mm_moe_routed_workspace_size(ctypes.byref(layer), t) if wsb is None else wsb
    return qs.lib.mm_moe_routed_f32(ctypes.byref(layer), x, ids, w, dst, t, ws, wsb, None)


def test_routed_refusals():
    assert qs.lib.mm_moe_routed_f32(None, X, XSC, XSC, DST, 1, WSP, 0, None) == NULL
    assert qs.lib.mm_moe_routed_workspace_size(None, 1) == 0
    for t in (qs.MM_TYPE_F32, qs.MM_TYPE_Q4_0, qs.MM_TYPE_Q8_0, 99):
        assert _moe(_layer(type=t)) == ARG
    for bad in (dict(D=48), dict(F=48), dict(D=0), dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=5), dict(D=2 ** 20 + 32)):
        assert _moe(_layer(**bad)) == SHAPE, bad
    assert _moe(_layer(), t=129) == SHAPE and _moe(_layer(), t=-1) == SHAPE
    assert _moe(_layer(), t=0, x=None, dst=None, ws=None) == OK
    for kind in (qs.MM_TYPE_MXFP4, qs.MM_TYPE_F8):
        for p in ("gate", "up", "down", "gate_scale", "up_scale", "down_scale"):
            assert _moe(_layer(type=kind, **{p: None})) == NULL, p
    for p in ("x", "dst", "ids", "w"):
        assert _moe(_layer(), **{p: None}) == NULL, p
    for p in ("gate", "up", "down"):
        assert _moe(_layer(**{p: getattr(_layer(), p) + 8})) == ALIGN, p
    assert _moe(_layer(up_scale=WSC + 2)) == ALIGN and _moe(_layer(), x=X + 4) == ALIGN and _moe(_layer(), ids=XSC + 2) == ALIGN
    assert _moe(_layer(), w=XSC + 1) == ALIGN and _moe(_layer(), ws=WSP + 64) == ALIGN
    need = qs.lib.mm_moe_routed_workspace_size(ctypes.byref(_layer()), 3)
    assert _moe(_layer(), wsb=need - 1) == WS and _moe(_layer(), ws=None) == WS
    # the router plays no part: neither its pointer nor its overlap
    assert _moe(_layer(router=DST + 4), wsb=need - 1) == WS
    for dst in (X + 3 * 256 * 4 - 4, W, W + G, W + 2 * G, WSC, WSC + G, WSC + 2 * G + 4 * 256 * 4 - 4, XSC, XSC + G, WSP):
        assert _moe(_layer(), dst=dst) == ALIAS, hex(dst)
    assert _moe(_layer(), ws=XSC) == ALIAS and _moe(_layer(), ws=X) == ALIAS


def test_the_layer_of_mxfp4_experts_with_a_router():
    def call(layer, dst=DST):
        size = qs.lib.mm_moe_workspace_size(ctypes.byref(layer), 3)
        return qs.lib.mm_moe_f32(ctypes.byref(layer), X, dst, None, None, 3, WSP, size, None)

    assert call(_layer()) == NULL                             # no router
    assert call(_layer(router=X + 8 * G, down_scale=None)) == NULL
    assert call(_layer(router=X + 8 * G), dst=WSC + 4 * 128 * 8 - 4) == ALIAS
    assert call(_layer(router=X + 8 * G), dst=W + 4 * 128 * 128 - 4) == ALIAS


def test_binding_refusals():
    import torch
    f32, u8, i32 = torch.float32, torch.uint8, torch.int32
    x = _as_gpu(2, 64, dtype=f32)
    cpu = torch.zeros((2, 64))
    w, ws = _as_gpu(7, 32, dtype=u8), _as_gpu(7, 4, dtype=u8)
    for f in (lambda: qs.quantize_mxfp4(cpu), lambda: qs.dequantize_mxfp4(cpu, cpu), lambda: qs.mul_mat_mxfp4_f32(w, ws, cpu),
              lambda: qs.mul_mat_mxfp4_f32(cpu, ws, x), lambda: qs.mul_mat_mxfp4_f32(None, ws, x),
              lambda: qs.mul_mat_mxfp4_f32(w, cpu, x), lambda: qs.rms_norm_f32(cpu), lambda: qs.rms_norm_f32(x, cpu),
              lambda: qs.route_f32(qs.Router(64, 2), cpu), lambda: qs.Router(64, 2, bias=torch.zeros(64)),
              lambda: qs.Router(64, 2, bias=3.0), lambda: qs.MoeLayer(qs.MM_TYPE_MXFP4, None, cpu, cpu, cpu, 32, 1),
              lambda: qs.mul_mat_mxfp4_mxfp4(w, ws, w.float(), ws)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: qs.mul_mat_mxfp4_f32(w, ws, _as_gpu(2, 96, dtype=f32)),
              lambda: qs.mul_mat_mxfp4_f32(w, _as_gpu(7, 2, dtype=u8), x),
              lambda: qs.mul_mat_mxfp4_mxfp4(w, ws, _as_gpu(2, 48, dtype=u8), _as_gpu(2, 4, dtype=u8)),
              lambda: qs.dequantize_mxfp4(w, ws, out=_as_gpu(7, 32, dtype=f32)),
              lambda: qs.quantize_mxfp4(x, out=(_as_gpu(2, 64, dtype=u8), _as_gpu(2, 4, dtype=u8))),
              lambda: qs.rms_norm_f32(x, _as_gpu(63, dtype=f32)), lambda: qs.rms_norm_f32(x, residual=_as_gpu(1, 64, dtype=f32)),
              lambda: qs.rms_norm_f32(x, out_type=qs.MM_TYPE_F16), lambda: qs.rms_norm_f32(x, out=_as_gpu(2, 32, dtype=f32)),
              lambda: qs.route_f32(qs.Router(63, 2), x), lambda: qs.route_f32(qs.Router(64, 2), x, ids=_as_gpu(2, 3, dtype=i32)),
              lambda: qs.Router(64, 2, score="max"), lambda: qs.Router(64, 2, bias=_as_gpu(63, dtype=f32)),
              lambda: qs.quantize_mxfp4(_as_gpu(64, 2, dtype=f32).t())):
        with pytest.raises(ValueError):
            f()


def test_layers_without_a_router():
    import torch
    e, d, f = 3, 64, 32
    u8 = torch.uint8
    w = [_as_gpu(e, n, k // 2, dtype=u8) for n, k in ((f, d), (f, d), (d, f))]
    s = [_as_gpu(e, n, 4, dtype=u8) for n in (f, f, d)]
    layer = qs.MoeLayer(qs.MM_TYPE_MXFP4, None, *w, f, 2, *s)
    assert (layer.e, layer.d, layer.struct.router) == (e, d, None) and layer.routed_workspace_size(3) > 0
    x = _as_gpu(2, d, dtype=torch.float32)
    with pytest.raises(ValueError):
        qs.moe_f32(layer, x)
    ids, weights = _as_gpu(2, 2, dtype=torch.int32), _as_gpu(2, 2, dtype=torch.float32)
    with pytest.raises(ValueError):
        qs.moe_routed_f32(layer, x, ids[:1], weights)
    with pytest.raises(TypeError):
        qs.moe_routed_f32(layer, x, ids.long(), weights)
    with pytest.raises(TypeError):
        qs.MoeLayer(qs.MM_TYPE_MXFP4, None, *w, f, 2)         # no scales
    with pytest.raises(ValueError):
        qs.MoeLayer(qs.MM_TYPE_MXFP4, None, *w, f, 2, *s, d=96)
    r = [_as_gpu(e, qs.repacked_bytes(n, k), dtype=u8) for n, k in ((f, d), (f, d), (d, f))]
    with pytest.raises(ValueError):
        qs.MoeLayer(qs.MM_TYPE_Q4_0R, None, *r, f, 2)         # D is in none of its tensors
    assert qs.MoeLayer(qs.MM_TYPE_Q4_0R, None, *r, f, 2, d=d).d == d
    assert qs.MoeLayer(qs.MM_TYPE_F16, None, *[_as_gpu(e, n, k, dtype=torch.float16) for n, k in ((f, d), (f, d), (d, f))], f, 1).d == d
