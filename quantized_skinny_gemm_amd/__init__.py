"""Python binding of libqsgemm.so, the gfx950 quantized skinny MUL_MAT library.

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI of ``include/mm.h``.  PyTorch supplies device
memory and the current stream.  Importing this package fails loudly when the
library has not been built (``python quantized_skinny_gemm_amd/build.py``);
there is no CPU fallback.

    dst = mul_mat_q4_0_f32(w_q4, x)      # w_q4: uint8 [N, K/32*18], x: f32 [M, K]
    dst = mul_mat_f16_f32(w_f16, x)      # w_f16: float16 [N, K]
    dst = mul_mat_f32(w_f32, x)          # w_f32: float32 [N, K]
    w_q4 = quantize_q4_0(w_f32)          # Q4_0 blocks of 18 bytes
    a_q8 = quantize_q8_0(x)              # Q8_0 blocks of 34 bytes (the wdata content)
    w_f8, w_scale = quantize_f8(w_f32, 128)       # e4m3 codes, a scale per 128 x 128 block
    dst = mul_mat_f8_f32(w_f8, w_scale, x)        # x quantized per row and 128 values within
    layer = MoeLayer(MM_TYPE_F16, router, gate, up, down, F, top_k)
    dst, ids, weights = moe_f32(layer, x)         # mixture-of-experts layer, a few tokens
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "LIB_PATH", "lib", "MM_TYPE_F32", "MM_TYPE_F16", "MM_TYPE_Q4_0", "MM_TYPE_Q8_0", "MM_TYPE_Q4_0R",
    "repacked_bytes", "repack_q4_0", "unpack_q4_0", "mul_mat_q4_0r_f32",
    "MMError", "quantize_q4_0", "quantize_q8_0", "mul_mat_q4_0_f32", "mul_mat_q8_0_f32",
    "mul_mat_f16_f32",
    "mul_mat_f32", "workspace_size", "debug_workspace_size", "row_bytes", "dispatch",
    "debug_mul_mat", "status_string", "q4_0_init", "q4_0_compute", "mul_mat_q4_0_f32_group",
    "group_workspace_size", "MM_TYPE_F8", "quantize_f8", "mul_mat_f8_f32", "mul_mat_f8_f8",
    "f8_workspace_size", "MoeLayer", "moe_f32",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqsgemm.so")

MM_TYPE_F32, MM_TYPE_F16, MM_TYPE_Q4_0, MM_TYPE_Q8_0, MM_TYPE_Q4_0R = 0, 1, 2, 3, 4
MM_TYPE_F8 = 5

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python quantized_skinny_gemm_amd/build.py` "
        "(the library has no CPU fallback)")

lib = ctypes.CDLL(LIB_PATH)

_i64, _sz, _vp, _int = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
for _name, _args, _res in [
    ("mm_quantize_q4_0", [_vp, _vp, _i64, _i64, _vp], _int),
    ("mm_quantize_q8_0", [_vp, _vp, _i64, _i64, _vp], _int),
    ("mm_mul_mat_q4_0_f32", [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_q4_0_f32_noalloc", [_vp, _vp, _vp, _i64, _i64, _i64, _vp], _int),
    ("mm_mul_mat_q4_0r_f32", [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_q8_0_f32", [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_repack_q4_0", [_vp, _vp, _i64, _i64, _vp], _int),
    ("mm_unpack_q4_0", [_vp, _vp, _i64, _i64, _vp], _int),
    ("mm_repacked_q4_0_bytes", [_i64, _i64], _i64),
    ("mm_mul_mat_f16_f32", [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_f32", [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_quantize_f8", [_vp, _vp, _vp, _i64, _i64, _int, _vp], _int),
    ("mm_mul_mat_f8_f32", [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_f8_f8", [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_f8_workspace_size", [_i64, _i64, _i64, _int], _sz),
    ("mm_moe_f32", [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp], _int),
    ("mm_moe_workspace_size", [_vp, _i64], _sz),
    ("mm_q4_0_init", [_vp, _vp, _i64, _i64, _i64, _sz, _vp], _int),
    ("mm_q4_0_compute", [_vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_q4_0_f32_group", [_int, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                   ctypes.POINTER(_i64), _vp, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_q4_0_group_workspace_size", [_int, ctypes.POINTER(_i64), _i64, _i64], _sz),
    ("mm_mul_mat_workspace_size", [_int, _i64, _i64, _i64], _sz),
    ("mm_debug_workspace_size", [_int, _i64, _i64, _i64, _int], _sz),
    ("mm_row_bytes", [_int, _i64], _i64),
    ("mm_status_string", [_int], ctypes.c_char_p),
    ("mm_dispatch", [_int, _i64, _i64, _i64, ctypes.POINTER(_int)], _int),
    ("mm_debug_mul_mat", [_int, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _vp,
                          _sz, _vp], _int),
]:
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class MMError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def status_string(status: int) -> str:
    return lib.mm_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MMError(status, what)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def row_bytes(mm_type: int, k: int) -> int:
    return int(lib.mm_row_bytes(int(mm_type), int(k)))


def workspace_size(mm_type: int, m: int, n: int, k: int) -> int:
    return int(lib.mm_mul_mat_workspace_size(int(mm_type), int(m), int(n), int(k)))


def debug_workspace_size(mm_type: int, m: int, n: int, k: int, variant: int) -> int:
    return int(lib.mm_debug_workspace_size(int(mm_type), int(m), int(n), int(k), int(variant)))


def dispatch(mm_type: int, m: int, n: int, k: int):
    """(variant, split, rows, cols, launches): the kernel mm_mul_mat_* picks at this shape."""
    out = (_int * 5)()
    _check(lib.mm_dispatch(int(mm_type), int(m), int(n), int(k), out), "mm_dispatch")
    return tuple(out)


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return None
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws


def _ptr(t):
    return None if t is None else t.data_ptr()


def quantize_q4_0(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """float32 [rows, K] -> uint8 [rows, K/32*18] Q4_0 blocks."""
    x = _dev(x, "x", torch.float32)
    rows, k = x.shape
    if out is None:
        out = torch.empty((rows, max(row_bytes(MM_TYPE_Q4_0, k), 0)), dtype=torch.uint8, device=x.device)
    _check(lib.mm_quantize_q4_0(_ptr(x), _ptr(out), rows, k, _stream(x)), "mm_quantize_q4_0")
    return out


def quantize_q8_0(x: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """float32 [rows, K] -> uint8 [rows, K/32*34] Q8_0 blocks."""
    x = _dev(x, "x", torch.float32)
    rows, k = x.shape
    if out is None:
        out = torch.empty((rows, max(row_bytes(MM_TYPE_Q8_0, k), 0)), dtype=torch.uint8, device=x.device)
    _check(lib.mm_quantize_q8_0(_ptr(x), _ptr(out), rows, k, _stream(x)), "mm_quantize_q8_0")
    return out


def _mul_mat(fn, mm_type, w, x, out, ws, what):
    m, k = x.shape
    n = w.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    else:
        _dev(out, "out", torch.float32)
    ws = _workspace(workspace_size(mm_type, m, n, k), x.device, ws)
    nbytes = 0 if ws is None else ws.numel()
    _check(fn(_ptr(w), _ptr(x), _ptr(out), m, n, k, _ptr(ws), nbytes, _stream(x)), what)
    return out


def mul_mat_q4_0_f32(w: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = Q8_0(x)[M, K] . Q4_0(w)[N, K]^T; w uint8 [N, K/32*18], x float32 [M, K]."""
    w = _dev(w, "w", torch.uint8)
    x = _dev(x, "x", torch.float32)
    if w.shape[1] != row_bytes(MM_TYPE_Q4_0, x.shape[1]):
        raise ValueError("w row bytes do not match K")
    return _mul_mat(lib.mm_mul_mat_q4_0_f32, MM_TYPE_Q4_0, w, x, out, ws, "mm_mul_mat_q4_0_f32")


def mul_mat_q8_0_f32(w: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = Q8_0(x)[M, K] . Q8_0(w)[N, K]^T; w uint8 [N, K/32*34], x float32 [M, K]."""
    w = _dev(w, "w", torch.uint8)
    x = _dev(x, "x", torch.float32)
    if w.shape[1] != row_bytes(MM_TYPE_Q8_0, x.shape[1]):
        raise ValueError("w row bytes do not match K")
    return _mul_mat(lib.mm_mul_mat_q8_0_f32, MM_TYPE_Q8_0, w, x, out, ws, "mm_mul_mat_q8_0_f32")


def repacked_bytes(n: int, k: int) -> int:
    return int(lib.mm_repacked_q4_0_bytes(int(n), int(k)))


def repack_q4_0(w: torch.Tensor, k: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """uint8 [N, K/32*18] Q4_0 -> uint8 [repacked_bytes(N, K)] repacked weights."""
    w = _dev(w, "w", torch.uint8)
    n = w.shape[0]
    if out is None:
        out = torch.empty(max(repacked_bytes(n, k), 0), dtype=torch.uint8, device=w.device)
    _check(lib.mm_repack_q4_0(_ptr(w), _ptr(out), n, k, _stream(w)), "mm_repack_q4_0")
    return out


def unpack_q4_0(wr: torch.Tensor, n: int, k: int, out: torch.Tensor | None = None) -> torch.Tensor:
    """Repacked weights -> uint8 [N, K/32*18] Q4_0."""
    wr = _dev(wr, "wr", torch.uint8)
    if out is None:
        out = torch.empty((n, max(row_bytes(MM_TYPE_Q4_0, k), 0)), dtype=torch.uint8, device=wr.device)
    _check(lib.mm_unpack_q4_0(_ptr(wr), _ptr(out), n, k, _stream(wr)), "mm_unpack_q4_0")
    return out


def mul_mat_q4_0r_f32(wr: torch.Tensor, n: int, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = Q8_0(x) . W^T with W (N x K) given in the repacked layout."""
    wr = _dev(wr, "wr", torch.uint8)
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    if wr.numel() < repacked_bytes(n, k):
        raise ValueError("repacked weights smaller than repacked_bytes(N, K)")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    else:
        _dev(out, "out", torch.float32)
    ws = _workspace(workspace_size(MM_TYPE_Q4_0R, m, n, k), x.device, ws)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib.mm_mul_mat_q4_0r_f32(_ptr(wr), _ptr(x), _ptr(out), m, n, k, _ptr(ws), nbytes,
                                    _stream(x)), "mm_mul_mat_q4_0r_f32")
    return out


def group_workspace_size(ns, m: int, k: int) -> int:
    arr = (_i64 * len(ns))(*ns)
    return int(lib.mm_mul_mat_q4_0_group_workspace_size(len(ns), arr, int(m), int(k)))


def mul_mat_q4_0_f32_group(ws_list, x: torch.Tensor, outs=None, ws=None):
    """[Q8_0(x) . Q4_0(w)^T for w in ws_list] as one grouped call (shared x); returns the outputs."""
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    ws_list = [_dev(w, f"w[{i}]", torch.uint8) for i, w in enumerate(ws_list)]
    for w in ws_list:
        if w.shape[1] != row_bytes(MM_TYPE_Q4_0, k):
            raise ValueError("w row bytes do not match K")
    ns = [w.shape[0] for w in ws_list]
    if outs is None:
        outs = [torch.empty((m, n), dtype=torch.float32, device=x.device) for n in ns]
    count = len(ws_list)
    src = (_vp * count)(*[w.data_ptr() for w in ws_list])
    dst = (_vp * count)(*[o.data_ptr() for o in outs])
    narr = (_i64 * count)(*ns)
    ws = _workspace(group_workspace_size(ns, m, k), x.device, ws)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib.mm_mul_mat_q4_0_f32_group(count, src, dst, narr, _ptr(x), m, k, _ptr(ws), nbytes,
                                         _stream(x)), "mm_mul_mat_q4_0_f32_group")
    return outs


def mul_mat_f16_f32(w: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = x[M, K] . w[N, K]^T; w float16, x float32."""
    w = _dev(w, "w", torch.float16)
    x = _dev(x, "x", torch.float32)
    if w.shape[1] != x.shape[1]:
        raise ValueError("K mismatch")
    return _mul_mat(lib.mm_mul_mat_f16_f32, MM_TYPE_F16, w, x, out, ws, "mm_mul_mat_f16_f32")


def mul_mat_f32(w: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = x[M, K] . w[N, K]^T; all float32."""
    w = _dev(w, "w", torch.float32)
    x = _dev(x, "x", torch.float32)
    if w.shape[1] != x.shape[1]:
        raise ValueError("K mismatch")
    return _mul_mat(lib.mm_mul_mat_f32, MM_TYPE_F32, w, x, out, ws, "mm_mul_mat_f32")


# ---- e4m3 products and the mixture-of-experts layer: calls of a few microseconds, so their checks are
# plain attribute comparisons, and sizes that only depend on the shape are computed once

def _public_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


# the same handle without a Stream object (a microsecond less); not in every build of torch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_F8_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _launch(fn, what: str, dev: int, *args) -> None:
    """fn(*args, current stream of device dev), with dev current during the call."""
    if dev == torch.cuda.current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != 0:
        raise MMError(status, what)


def _on(t, name: str, shape, dtypes, dev: int) -> None:
    """t is a contiguous GPU tensor of this shape, one of dtypes, on device dev."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {dtypes[0]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


_F32 = (torch.float32,)


def _ceil128(v: int) -> int:
    return (v + 127) // 128


def quantize_f8(x: torch.Tensor, block_rows: int = 1, out=None):
    """float32 [rows, K] -> (codes float8_e4m3fn [rows, K], scales float32
    [ceil(rows / block_rows), ceil(K / 128)]); block_rows 1 (activations) or 128 (weights)."""
    x = _dev(x, "x", torch.float32)
    rows, k = x.shape
    nb = rows if block_rows == 1 else _ceil128(rows)
    dev = x.get_device()
    if out is None:
        codes = torch.empty((rows, k), dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty((nb, _ceil128(k)), dtype=torch.float32, device=x.device)
    else:
        codes, scales = out
        _on(codes, "out codes", (rows, k), _F8_DTYPES, dev)
        _on(scales, "out scales", (nb, _ceil128(k)), _F32, dev)
    _launch(lib.mm_quantize_f8, "mm_quantize_f8", dev, x.data_ptr(), codes.data_ptr(), scales.data_ptr(),
            rows, k, block_rows)
    return codes, scales


@functools.lru_cache(maxsize=4096)
def f8_workspace_size(m: int, n: int, k: int, src1_quantized: bool = False) -> int:
    return int(lib.mm_mul_mat_f8_workspace_size(int(m), int(n), int(k), int(src1_quantized)))


def _f8_weights(w, w_scale, k: int, dev: int) -> int:
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("w must be a 2-d GPU (HIP) tensor")
    n = w.shape[0]
    _on(w, "w", (n, k), _F8_DTYPES, dev)
    _on(w_scale, "w_scale", (_ceil128(n), _ceil128(k)), _F32, dev)
    return n


def _buffers(m, n, device, dev, out, need, ws):
    """out (allocated if None, checked otherwise) and the workspace with its size."""
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=device)
    else:
        _on(out, "out", (m, n), _F32, dev)
    if need == 0:
        return out, None, 0
    if ws is None or ws.numel() < need:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    elif not ws.is_cuda or ws.get_device() != dev or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{dev}")
    return out, ws, ws.numel()


def mul_mat_f8_f32(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = F8(x)[M, K] . F8(w)[N, K]^T; w e4m3 [N, K] with scales [ceil(N/128), ceil(K/128)],
    x float32 [M, K], quantized within (one scale per row and 128 values)."""
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    dev = x.get_device()
    n = _f8_weights(w, w_scale, k, dev)
    out, ws, nbytes = _buffers(m, n, x.device, dev, out, f8_workspace_size(m, n, k, False), ws)
    _launch(lib.mm_mul_mat_f8_f32, "mm_mul_mat_f8_f32", dev, w.data_ptr(), w_scale.data_ptr(), x.data_ptr(),
            out.data_ptr(), m, n, k, None if ws is None else ws.data_ptr(), nbytes)
    return out


def mul_mat_f8_f8(w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, a_scale: torch.Tensor,
                  out=None, ws=None) -> torch.Tensor:
    """mul_mat_f8_f32 with src1 quantized already: a e4m3 [M, K], a_scale [M, ceil(K/128)]
    (quantize_f8 with block_rows 1)."""
    a = _dev(a, "a")
    m, k = a.shape
    dev = a.get_device()
    _on(a, "a", (m, k), _F8_DTYPES, dev)
    _on(a_scale, "a_scale", (m, _ceil128(k)), _F32, dev)
    n = _f8_weights(w, w_scale, k, dev)
    out, ws, nbytes = _buffers(m, n, a.device, dev, out, f8_workspace_size(m, n, k, True), ws)
    _launch(lib.mm_mul_mat_f8_f8, "mm_mul_mat_f8_f8", dev, w.data_ptr(), w_scale.data_ptr(), a.data_ptr(),
            a_scale.data_ptr(), out.data_ptr(), m, n, k, None if ws is None else ws.data_ptr(), nbytes)
    return out


class _MoeStruct(ctypes.Structure):
    _fields_ = [("type", _int), ("top_k", _int), ("norm", _int), ("D", _i64), ("F", _i64), ("E", _i64),
                ("router", _vp), ("gate", _vp), ("up", _vp), ("down", _vp),
                ("gate_scale", _vp), ("up_scale", _vp), ("down_scale", _vp)]


_MOE_POINTERS = ("router", "gate", "up", "down", "gate_scale", "up_scale", "down_scale")
_MOE_DTYPES = {MM_TYPE_Q4_0R: (torch.uint8,), MM_TYPE_F8: _F8_DTYPES, MM_TYPE_F16: (torch.float16,)}


class MoeLayer:
    """The weights of a mixture-of-experts layer, for moe_f32 (holds the tensors and the C struct, whose
    addresses are the tensors' own at each call).

    router float32 [E, D]; gate, up (F x D per expert) and down (D x F) by mm_type:
    MM_TYPE_Q4_0R uint8 [E, repacked_bytes(rows, K)] (repack_q4_0 of each expert), MM_TYPE_F8
    e4m3 [E, rows, K] with float32 scales [E, ceil(rows/128), ceil(K/128)], MM_TYPE_F16 float16
    [E, rows, K].  norm: the top_k probabilities are divided by their sum."""

    def __init__(self, mm_type, router, gate, up, down, f, top_k, gate_scale=None, up_scale=None,
                 down_scale=None, norm=True):
        _dev(router, "router", torch.float32)
        e, d = router.shape
        f, top_k = int(f), int(top_k)
        if mm_type not in _MOE_DTYPES:
            raise ValueError("mm_type must be MM_TYPE_Q4_0R, MM_TYPE_F8 or MM_TYPE_F16")
        scales = (gate_scale, up_scale, down_scale) if mm_type == MM_TYPE_F8 else (None,) * 3
        self.dev, self.device, self.d, self.f, self.e, self.top_k = router.get_device(), router.device, d, f, e, top_k
        self.tensors = (router, gate, up, down, *scales)
        self.struct = _MoeStruct(mm_type, top_k, int(bool(norm)), d, f, e)
        self._ref = ctypes.byref(self.struct)
        self._sizes = {}
        self._live = [(t.data_ptr, t.stride) for t in self.tensors if isinstance(t, torch.Tensor)]
        self._seen = None
        self._take()

    def _take(self):
        """The C struct, with the addresses that the tensors have now: a weight that was given other
        storage or strides since the last call (t.data = ..., set_, a resize) is checked again."""
        seen = [f() for get in self._live for f in get]
        if seen != self._seen:
            kind, d, f, e, dev = self.struct.type, self.d, self.f, self.e, self.dev
            router, *rest = self.tensors
            _on(router, "router", (e, d), _F32, dev)
            for name, w, scale, rows, k in zip(("gate", "up", "down"), rest[:3], rest[3:], (f, f, d), (d, d, f)):
                _on(w, name, (e, repacked_bytes(rows, k)) if kind == MM_TYPE_Q4_0R else (e, rows, k),
                    _MOE_DTYPES[kind], dev)
                if kind == MM_TYPE_F8:
                    _on(scale, f"{name}_scale", (e, _ceil128(rows), _ceil128(k)), _F32, dev)
            for field, t in zip(_MOE_POINTERS, self.tensors):
                setattr(self.struct, field, _ptr(t))
            self._seen = seen
        return self._ref

    def workspace_size(self, t: int) -> int:
        """Bytes of workspace for t tokens (0: t is out of range, or the layer's sizes are)."""
        if t not in self._sizes:
            self._sizes[t] = int(lib.mm_moe_workspace_size(self._ref, int(t)))
        return self._sizes[t]


_I32 = (torch.int32,)


def moe_f32(layer: MoeLayer, x: torch.Tensor, out=None, ids=None, weights=None, ws=None):
    """(dst [T, D], ids int32 [T, top_k], weights [T, top_k]) of the layer on x float32 [T, D]."""
    x = _dev(x, "x", torch.float32)
    t = x.shape[0]
    dev, k = layer.dev, layer.top_k
    _on(x, "x", (t, layer.d), _F32, dev)
    if ids is None:
        ids = torch.empty((t, k), dtype=torch.int32, device=layer.device)
    else:
        _on(ids, "ids", (t, k), _I32, dev)
    if weights is None:
        weights = torch.empty((t, k), dtype=torch.float32, device=layer.device)
    else:
        _on(weights, "weights", (t, k), _F32, dev)
    out, ws, nbytes = _buffers(t, layer.d, layer.device, dev, out, layer.workspace_size(t), ws)
    _launch(lib.mm_moe_f32, "mm_moe_f32", dev, layer._take(), x.data_ptr(), out.data_ptr(), ids.data_ptr(),
            weights.data_ptr(), t, None if ws is None else ws.data_ptr(), nbytes)
    return out, ids, weights


def q4_0_init(x: torch.Tensor, n: int, ws: torch.Tensor | None = None) -> torch.Tensor:
    """INIT stage: quantize x (float32 [M, K]) to Q8_0 into a workspace sized for
    (M, n, K); returns the workspace for q4_0_compute."""
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    need = workspace_size(MM_TYPE_Q4_0, m, n, k)
    ws = _workspace(need, x.device, ws)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib.mm_q4_0_init(_ptr(x), _ptr(ws), m, n, k, nbytes, _stream(x)), "mm_q4_0_init")
    return ws


def q4_0_compute(w: torch.Tensor, ws: torch.Tensor, m: int, k: int, out=None) -> torch.Tensor:
    """COMPUTE stage: dst[M, N] from the Q8_0 wdata a q4_0_init with the same (M, N, K) left in ws."""
    w = _dev(w, "w", torch.uint8)
    n = w.shape[0]
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=w.device)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib.mm_q4_0_compute(_ptr(w), _ptr(out), m, n, k, _ptr(ws), nbytes, _stream(w)),
           "mm_q4_0_compute")
    return out


_W_DTYPE = {MM_TYPE_Q4_0: torch.uint8, MM_TYPE_F16: torch.float16, MM_TYPE_F32: torch.float32}


def debug_mul_mat(mm_type: int, w: torch.Tensor, x: torch.Tensor, variant: int = 0,
                  n0: int = 0, n1: int = 0):
    """Product with the kernel forced (0 auto, 1 narrow, 2 wide, 3 skinny MFMA); for Q4_0
    also the int32 block dots [M, n1-n0, K/32] of columns n0..n1-1 as written by the
    production kernel."""
    w = _dev(w, "w", _W_DTYPE[mm_type])
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    n = w.shape[0]
    out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    dots = None
    if mm_type == MM_TYPE_Q4_0 and n1 > n0:
        dots = torch.empty((m, n1 - n0, k // 32), dtype=torch.int32, device=x.device)
    ws = _workspace(debug_workspace_size(mm_type, m, n, k, variant), x.device, None)
    nbytes = 0 if ws is None else ws.numel()
    _check(lib.mm_debug_mul_mat(mm_type, _ptr(w), _ptr(x), _ptr(out), _ptr(dots), m, n, k, n0,
                                n1, variant, _ptr(ws), nbytes, _stream(x)), "mm_debug_mul_mat")
    return out, dots
