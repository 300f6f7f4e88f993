"""Host-side checks of the e4m3 and mixture-of-experts entry points: arguments are refused before any HIP call
(the pointers here are never dereferenced), workspace sizes, the binding's own checks."""
from __future__ import annotations

import ctypes

import pytest

import quantized_skinny_gemm_amd as qs
from tests import plans

OK, NULL, SHAPE, ALIGN, WS, ALIAS, ARG = 0, -1, -2, -3, -4, -5, -8
W, WSC, X, XSC, DST, WSP = (0x7f0000000000 + (i << 36) for i in range(6))
G = 1 << 30


def _f32(m=4, n=256, k=512, w=W, wsc=WSC, x=X, dst=DST, ws=WSP, wsb=None):
    wsb = qs.f8_workspace_size(m, n, k) if wsb is None else wsb
    return qs.lib.mm_mul_mat_f8_f32(w, wsc, x, dst, m, n, k, ws, wsb, None)


def _f8(m=4, n=256, k=512, w=W, wsc=WSC, x=X, xsc=XSC, dst=DST, ws=WSP, wsb=None):
    wsb = qs.f8_workspace_size(m, n, k, True) if wsb is None else wsb
    return qs.lib.mm_mul_mat_f8_f8(w, wsc, x, xsc, dst, m, n, k, ws, wsb, None)


def test_type_and_sizes():
    assert qs.MM_TYPE_F8 == 5
    assert qs.row_bytes(qs.MM_TYPE_F8, 4096) == 4096
    assert qs.row_bytes(qs.MM_TYPE_F8, 48) == -1
    assert qs.workspace_size(qs.MM_TYPE_F8, 100, 300, 512) == qs.f8_workspace_size(100, 300, 512)
    # src1 as codes needs no more than src1 as f32
    for m, n, k in ((1, 4096, 4096), (16, 14336, 4096), (128, 4096, 14336), (512, 14336, 4096)):
        assert qs.f8_workspace_size(m, n, k, True) <= qs.f8_workspace_size(m, n, k)
    assert qs.f8_workspace_size(-1, 4, 32) == 0 and qs.f8_workspace_size(1, 4, 33) == 0
    # the type has entry points of its own
    assert qs.lib.mm_dispatch(qs.MM_TYPE_F8, 1, 64, 64, None) == ARG
    assert qs.lib.mm_debug_mul_mat(qs.MM_TYPE_F8, W, X, DST, None, 1, 64, 64, 0, 0, 0, None, 0, None) == ARG


@pytest.mark.parametrize("call", [_f32, _f8])
def test_product_refusals(call):
    for bad in (dict(k=48), dict(m=-1), dict(n=-1), dict(k=-32), dict(n=2 ** 31), dict(m=2 ** 31), dict(k=2 ** 23 + 32)):
        assert call(**{**dict(wsb=0), **bad}) == SHAPE, bad
    for p in ("w", "wsc", "x", "dst"):
        assert call(**{p: None}) == NULL, p
    assert call(w=W + 8) == ALIGN and call(wsc=WSC + 2) == ALIGN and call(x=X + 4) == ALIGN and call(dst=DST + 2) == ALIGN
    assert call(dst=W + 4096) == ALIAS and call(dst=X) == ALIAS and call(dst=WSC) == ALIAS
    # empty products look at no pointer
    assert call(m=0, w=None, x=None, dst=None, wsb=0) == OK and call(n=0, w=None, dst=None, wsb=0) == OK


@pytest.mark.parametrize("call", [_f32, _f8])
def test_product_refuses_what_no_grid_covers(call):
    # tile ends past 2^31, launches of 2^32 threads and more
    for m, n, k in ((1, 2 ** 31 - 1, 32), (2 ** 31 - 1, 1, 32), (8, 2 ** 28, 4128), (2 ** 23, 2 ** 15, 32),
                    (2 ** 17, 2 ** 22, 32)):
        assert call(m, n, k, wsb=0) == SHAPE, (m, n, k)


def test_workspace_of_few_rows():
    # f32 rows that the product quantizes within need no workspace; the same rows as codes may
    assert qs.f8_workspace_size(9, 9400, 3584) == 0 < qs.f8_workspace_size(9, 9400, 3584, True)
    assert _f8(9, 9400, 3584, ws=None, wsb=0) == WS


def test_product_workspace_refusals():
    m, n, k = 100, 256, 4096
    need = qs.f8_workspace_size(m, n, k)
    assert need >= m * k + 4 * m * 32
    assert _f32(m, n, k, wsb=need - 1) == WS and _f32(m, n, k, ws=None) == WS
    assert _f32(m, n, k, ws=WSP + 64) == ALIGN
    for p in (W, WSC, X, DST):
        assert _f32(m, n, k, ws=p) == ALIAS
    assert _f8(m, n, k, xsc=None) == NULL and _f8(m, n, k, xsc=XSC + 1) == ALIGN
    assert _f8(m, n, k, dst=XSC) == ALIAS


def test_quantize_refusals():
    q = qs.lib.mm_quantize_f8
    assert q(X, W, WSC, 4, 64, 2, None) == ARG
    assert q(X, W, WSC, 4, 48, 1, None) == SHAPE and q(X, W, WSC, -1, 64, 1, None) == SHAPE
    assert q(X, W, WSC, 4, 2 ** 23 + 32, 128, None) == SHAPE
    for i in range(3):
        p = [X, W, WSC]
        p[i] = None
        assert q(*p, 4, 64, 1, None) == NULL
    assert q(X + 4, W, WSC, 4, 64, 1, None) == ALIGN and q(X, W + 8, WSC, 4, 64, 1, None) == ALIGN
    assert q(X, W, WSC + 2, 4, 64, 128, None) == ALIGN
    assert q(X, X + 256, WSC, 4, 64, 1, None) == ALIAS and q(X, W, X + 16, 4, 64, 1, None) == ALIAS
    assert q(X, W, W, 4, 64, 1, None) == ALIAS
    assert q(None, None, None, 0, 64, 1, None) == OK and q(None, None, None, 3, 0, 128, None) == OK


class _L(qs._MoeStruct):
    pass


def _layer(**kw):
    base = dict(type=qs.MM_TYPE_F8, top_k=2, norm=1, D=256, F=128, E=4, router=X + 8 * G, gate=W, up=W + G, down=W + 2 * G,
                gate_scale=WSC, up_scale=WSC + G, down_scale=WSC + 2 * G)
    base.update(kw)
    return qs._MoeStruct(**base)


def _moe(layer, t=3, x=X, dst=DST, ids=None, weights=None, ws=WSP, wsb=None):
    wsb = qs.lib.mm_moe_workspace_size(ctypes.byref(layer), t) if wsb is None else wsb
    return qs.lib.mm_moe_f32(ctypes.byref(layer), x, dst, ids, weights, t, ws, wsb, None)


def test_moe_refusals():
    assert qs.lib.mm_moe_f32(None, X, DST, None, None, 1, WSP, 0, None) == NULL
    assert qs.lib.mm_moe_workspace_size(None, 1) == 0
    for t in (qs.MM_TYPE_F32, qs.MM_TYPE_Q4_0, qs.MM_TYPE_Q8_0, 99):
        assert _moe(_layer(type=t)) == ARG
    for bad in (dict(D=48), dict(F=48), dict(D=0), dict(F=0), dict(E=0), dict(E=513), dict(top_k=0), dict(top_k=5),
                dict(top_k=17, E=64), dict(D=2 ** 20 + 32), dict(F=2 ** 20 + 32)):
        assert _moe(_layer(**bad)) == SHAPE, bad
    assert _moe(_layer(), t=129) == SHAPE and _moe(_layer(), t=-1) == SHAPE
    assert _moe(_layer(), t=0, x=None, dst=None, ws=None) == OK
    for p in ("router", "gate", "up", "down", "gate_scale", "up_scale", "down_scale"):
        assert _moe(_layer(**{p: None})) == NULL, p
    assert _moe(_layer(), x=None) == NULL and _moe(_layer(), dst=None) == NULL
    for p in ("router", "gate", "up", "down"):
        assert _moe(_layer(**{p: getattr(_layer(), p) + 8})) == ALIGN, p
    assert _moe(_layer(gate_scale=WSC + 2)) == ALIGN
    assert _moe(_layer(), x=X + 4) == ALIGN and _moe(_layer(), dst=DST + 1) == ALIGN
    assert _moe(_layer(), ids=DST + G + 2) == ALIGN and _moe(_layer(), ws=WSP + 64) == ALIGN
    need = qs.lib.mm_moe_workspace_size(ctypes.byref(_layer()), 3)
    assert _moe(_layer(), wsb=need - 1) == WS and _moe(_layer(), ws=None) == WS


def test_moe_aliasing():
    x_bytes, k_bytes = 3 * 256 * 4, 3 * 2 * 4
    for dst in (X + x_bytes - 4, W, W + G, W + 2 * G, WSC, WSC + G, WSC + 2 * G, X + 8 * G, WSP):
        assert _moe(_layer(), dst=dst) == ALIAS
    assert _moe(_layer(), ids=DST + 4) == ALIAS and _moe(_layer(), weights=X) == ALIAS
    assert _moe(_layer(), ids=DST + G, weights=DST + G + k_bytes - 4) == ALIAS
    assert _moe(_layer(), ws=DST) == ALIAS and _moe(_layer(), ws=W) == ALIAS


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros((2, 64))
    for f in (lambda: qs.quantize_f8(x), lambda: qs.mul_mat_f8_f32(x, x, x), lambda: qs.mul_mat_f8_f8(x, x, x, x),
              lambda: qs.MoeLayer(qs.MM_TYPE_F16, x, x, x, x, 32, 1)):
        with pytest.raises(TypeError):
            f()


def _as_gpu(*shape, dtype):
    """A tensor in host memory that the binding takes for one on GPU 0 (no call here reaches the GPU)."""
    import torch

    class Fake(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

    return torch.zeros(shape, dtype=dtype).as_subclass(Fake)


def _fake_layer(kind, d=64, f=32, e=3):
    import torch
    if kind == qs.MM_TYPE_Q4_0R:
        w = [_as_gpu(e, qs.repacked_bytes(n, k), dtype=torch.uint8) for n, k in ((f, d), (f, d), (d, f))]
    else:
        dtype = torch.float16 if kind == qs.MM_TYPE_F16 else torch.uint8
        w = [_as_gpu(e, n, k, dtype=dtype) for n, k in ((f, d), (f, d), (d, f))]
    scales = [_as_gpu(e, 1, 1, dtype=torch.float32) for _ in range(3)] if kind == qs.MM_TYPE_F8 else [None] * 3
    return qs.MoeLayer(kind, _as_gpu(e, d, dtype=torch.float32), *w, f, 2, *scales)


@pytest.mark.parametrize("kind", [qs.MM_TYPE_Q4_0R, qs.MM_TYPE_F8, qs.MM_TYPE_F16])
def test_layer_follows_its_tensors_to_other_storage(kind, monkeypatch):
    """A weight given other storage after the layer was made: the next call reads that one, or refuses it; the
    address of the freed storage is never passed on."""
    import torch
    layer = _fake_layer(kind)
    x = _as_gpu(2, 64, dtype=torch.float32)
    sent = []

    def launch(fn, what, dev, ref, *args):
        sent.append([getattr(layer.struct, n) for n, _ in qs._MoeStruct._fields_[6:]])
        assert ref is layer._ref

    monkeypatch.setattr(qs, "_launch", launch)
    bufs = dict(out=_as_gpu(2, 64, dtype=torch.float32), ids=_as_gpu(2, 2, dtype=torch.int32),
                weights=_as_gpu(2, 2, dtype=torch.float32), ws=_as_gpu(layer.workspace_size(2), dtype=torch.uint8))
    now = lambda: [None if t is None else t.data_ptr() for t in layer.tensors]
    qs.moe_f32(layer, x, **bufs)
    assert sent[-1] == now()
    for i, t in enumerate(layer.tensors):
        if t is None:
            continue
        kept = t.data                                     # the first storage lives on, so addresses differ
        t.data = torch.ones_like(kept)
        assert t.data_ptr() != kept.data_ptr()
        qs.moe_f32(layer, x, **bufs)
        assert sent[-1] == now(), i
        t.resize_((t.shape[0] + 1, *t.shape[1:]))
        with pytest.raises(ValueError):
            qs.moe_f32(layer, x, **bufs)
        t.data = torch.zeros(kept.shape, dtype=torch.float64)
        with pytest.raises(TypeError):
            qs.moe_f32(layer, x, **bufs)
        t.data = kept
        qs.moe_f32(layer, x, **bufs)
        assert sent[-1] == now(), i
    if kind == qs.MM_TYPE_F16:                            # the same storage, read another way
        gate = layer.tensors[1]
        gate.transpose_(1, 2)
        with pytest.raises(ValueError):
            qs.moe_f32(layer, x, **bufs)
        gate.transpose_(1, 2)
        qs.moe_f32(layer, x, **bufs)


def test_layer_refuses_what_is_no_tensor():
    import torch
    r = _as_gpu(3, 64, dtype=torch.float32)
    w = _as_gpu(3, 32, 64, dtype=torch.float16)
    for bad in (None, [1, 2], 3.0):
        with pytest.raises(TypeError):
            qs.MoeLayer(qs.MM_TYPE_F16, r, w, bad, w, 32, 2)


def test_binding_loads_without_the_private_stream_query():
    """A build of torch that lacks the private name: everything loads, streams come from the public call."""
    import subprocess
    import sys
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import quantized_skinny_gemm_amd as qs\n"
            "assert qs._raw_stream is qs._public_stream\n"
            "print(qs.workspace_size(qs.MM_TYPE_Q4_0, 5, 64, 64), qs.f8_workspace_size(100, 256, 4096))\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120,
                       cwd=__file__.rsplit("/tests/", 1)[0])
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [str(qs.workspace_size(qs.MM_TYPE_Q4_0, 5, 64, 64)), str(qs.f8_workspace_size(100, 256, 4096))]


@pytest.mark.parametrize("m,n,k,given,kind", [
    # one row, K below 4096: the kernel that measures faster at each size
    (1, 18944, 3584, False, "fused"), (8, 18944, 3584, False, "fused"), (1, 65536, 3584, False, "fused"),
    (1, 152064, 2560, False, "fused"), (1, 24000, 2048, False, "fused"), (1, 30000, 2048, False, "wide"),
    (1, 12500, 1024, False, "wide"), (1, 65536, 2304, False, "wide"), (1, 12000, 1024, False, "fused"),
    (1, 8192, 1024, True, "skinny"), (16, 8192, 3200, True, "skinny"), (1, 8200, 1024, True, "wide"),
    (4, 18944, 3584, True, "skinny"), (8, 24000, 2816, True, "wide"), (1, 18944, 2560, True, "wide"),
    (8, 65536, 4096, True, "skinny"), (9, 65536, 4096, True, "wide"),
])
def test_kernel_of_a_few_rows(m, n, k, given, kind):
    assert plans.f8(m, n, k, given).kind == kind


@pytest.mark.parametrize("m,n,k,given,kind", [
    # few weight rows, long K: the kernel that splits K over the CUs
    (16, 1024, 14336, True, "wide"), (4, 1024, 14336, True, "wide"), (16, 1024, 14336, False, "wide"),
    (1, 1024, 28672, True, "wide"), (4, 40, 131072, False, "wide"), (16, 2048, 8192, True, "wide"),
    (8, 2048, 8192, True, "skinny"), (24, 1024, 4096, True, "skinny"), (8, 4096, 14336, True, "skinny"),
    # a second tile of 16 src1 rows, over and up to 4096 weight rows
    (24, 8192, 1024, True, "wide"), (24, 7000, 3200, True, "wide"), (16, 7000, 3200, True, "skinny"),
    (24, 4096, 4096, True, "skinny"), (24, 3200, 8192, True, "wide"), (16, 3200, 8192, True, "skinny"),
])
def test_kernel_of_a_few_rows_on_few_weight_rows(m, n, k, given, kind):
    assert plans.f8(m, n, k, given).kind == kind


def test_few_row_kernels_hold_all_rows_of_src1():
    """The skinny kernel has no second pass over src1 rows, the fused one 16 rows and the LDS of a workgroup."""
    for m in range(1, 40):
        for n in (16, 1000, 2049, 4096, 4097, 8192, 8193, 60000):
            for k in (32, 1056, 2048, 2720, 4096, 8192, 14336, 65536):
                for given in (False, True):
                    p = plans.f8(m, n, k, given)
                    assert p.kind != "skinny" or m <= 16 * p.nt, (m, n, k, given)
                    assert p.kind != "fused" or m <= 16 and m * -(-k // 128) <= 32 * p.nt, (m, n, k, given)


@pytest.mark.parametrize("kind", [qs.MM_TYPE_Q4_0R, qs.MM_TYPE_F8, qs.MM_TYPE_F16])
@pytest.mark.parametrize("dim", ["D", "F"])
def test_moe_width_limit(kind, dim):
    """2^18 is the last width: split h of 128 tokens on 16 experts is 2^31 bytes there, offsets are 32 bits."""
    size = lambda width: qs.lib.mm_moe_workspace_size(ctypes.byref(_layer(type=kind, E=16, top_k=16, **{dim: width})), 128)
    assert size(2 ** 18) > 2048 * (4 * 2 ** 18 if dim == "F" else 4 * 128)
    for width in (2 ** 18 + 32, 2 ** 19, 2 ** 20):
        assert size(width) == 0 and _moe(_layer(type=kind, **{dim: width}), wsb=0) == SHAPE


def _gpu_shapes():
    from tests import test_gpu_f8 as t
    listed = next(m.args[1] for m in t.test_products.pytestmark if m.name == "parametrize")
    return listed, t.PLANNED


def _kind_of_plan(m, n, k, given):
    p, tail = plans.f8(m, n, k, given), k % 128 != 0
    if p.kind != "wide":
        return p.kind, p.nt, tail
    uneven = p.split > 1 and -(-k // 128) % p.kchunk != 0
    return p.bm, p.bn, p.split > 1, uneven, tail


def test_gpu_shapes_have_the_plans_that_they_are_listed_for():
    for shape, want in _gpu_shapes()[1]:
        p = plans.f8(*shape)
        if want[0] in ("fused", "skinny"):
            assert (p.kind, p.nt) == want, shape
        else:
            assert (p.bm, p.bn, p.split, p.kchunk) == want and p == plans.f8(*shape, True), shape


def test_gpu_shapes_meet_every_kind_of_plan():
    """Kernel, rounds or tile, K slices even, uneven or one, K ending inside a block or not: whatever the plan gives on a
    wide grid of calls, a tested shape has it."""
    listed, planned = _gpu_shapes()
    tested = {_kind_of_plan(*s, g) for s in [*listed, *(s for s, _ in planned)] for g in (False, True)}
    for m in (1, 2, 3, 5, 8, 9, 16, 17, 24, 25, 64, 65, 128, 129, 256, 257, 300, 512, 1100, 2048):
        for n in (16, 300, 1000, 2049, 4096, 5000, 8192, 8200, 12500, 33000, 130000):
            for k in (32, 128, 160, 1024, 1056, 2080, 2560, 3584, 4096, 4128, 8192, 8224, 11008, 14336, 28672, 32992):
                for given in (False, True):
                    assert _kind_of_plan(m, n, k, given) in tested, (m, n, k, given, plans.f8(m, n, k, given))


def test_gpu_layers_have_the_plans_that_they_are_listed_for():
    from tests import test_gpu_moe as t
    kinds = {"q4_0r": qs.MM_TYPE_Q4_0R, "f8": qs.MM_TYPE_F8, "f16": qs.MM_TYPE_F16}
    d, f, e, k = (t.LONG[n] for n in ("d", "f", "e", "top_k"))
    for tokens, by_kind in t.LONG_PLANS.items():
        for kind, want in by_kind.items():
            p = plans.moe(kinds[kind], tokens, d, f, e, k)
            assert (p.rt, p.slices) == want, (tokens, kind, p)
            # units of 128 k for 8 waves: not the same number each; several groups of 32 rows per workgroup
            assert -(-d // 128) > 16 and -(-d // 128) % 8 and p.up_groups < f // 32, (tokens, kind, p)
            assert p.fold
    assert all(plans.moe(v, 70, 96, 16416, 2, 2)[2:] == (1, 4) for v in kinds.values())
    for e in (300, 200, 512):
        assert not plans.moe(qs.MM_TYPE_F8, {300: 1, 200: 2, 512: 4}[e], 96, 64, e, 1).fold
