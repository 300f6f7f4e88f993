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
    w_mx, w_scale = quantize_mxfp4(w_f32)         # 4-bit codes, a power of two per 32 values
    dst = mul_mat_mxfp4_f32(w_mx, w_scale, x)     # x quantized to MXFP4 within
    (a, a_scale), h = rms_norm_f32(x, g, residual=h, out_type=MM_TYPE_MXFP4)
    dst = mul_mat_mxfp4_mxfp4(w_mx, w_scale, a, a_scale)
    ids, weights = route_f32(Router(E, top_k, score="sigmoid", bias=b, groups=8, group_k=4), logits)
    dst = moe_routed_f32(layer, x, ids, weights)  # the layer's experts for that choice
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
    "f8_workspace_size", "MoeLayer", "moe_f32", "MM_TYPE_MXFP4", "quantize_mxfp4", "dequantize_mxfp4",
    "mul_mat_mxfp4_f32", "mul_mat_mxfp4_mxfp4", "mxfp4_workspace_size", "rms_norm_f32", "Router",
    "route_f32", "moe_routed_f32",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqsgemm.so")

MM_TYPE_F32, MM_TYPE_F16, MM_TYPE_Q4_0, MM_TYPE_Q8_0, MM_TYPE_Q4_0R = 0, 1, 2, 3, 4
MM_TYPE_F8 = 5
MM_TYPE_MXFP4 = 6

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
    ("mm_quantize_mxfp4", [_vp, _vp, _vp, _i64, _i64, _vp], _int),
    ("mm_dequantize_mxfp4", [_vp, _vp, _vp, _i64, _i64, _vp], _int),
    ("mm_mul_mat_mxfp4_f32", [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_mxfp4_mxfp4", [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp], _int),
    ("mm_mul_mat_mxfp4_workspace_size", [_i64, _i64, _i64, _int], _sz),
    ("mm_rms_norm_f32", [_vp, _vp, _vp, ctypes.c_float, _vp, _int, _vp, _vp, _i64, _i64, _vp], _int),
    ("mm_route_f32", [_vp, _vp, _vp, _vp, _i64, _vp], _int),
    ("mm_moe_routed_f32", [_vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp], _int),
    ("mm_moe_routed_workspace_size", [_vp, _i64], _sz),
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
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_F8_DTYPES = (torch.float8_e4m3fn, torch.uint8)


def _launch(fn, what: str, dev: int, *args) -> None:
    """fn(*args, current stream of device dev), with dev current during the call."""
    if dev == _current_device():
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != 0:
        raise MMError(status, what)


def _on(t, name: str, shape, dtypes, dev: int) -> None:
    """t is a contiguous GPU tensor of this shape, one of dtypes, on device dev."""
    if type(t) is torch.Tensor and t.dtype in dtypes and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
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


def _new(rows: int, cols: int, dtype, device):
    """An uninitialised tensor [rows, cols] (torch.empty takes half a microsecond longer)."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


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
        codes = _new(rows, k, torch.float8_e4m3fn, x.device)
        scales = _new(nb, _ceil128(k), torch.float32, x.device)
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
        out = _new(m, n, torch.float32, device)
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


# MXFP4 codes are pairs in bytes, its scales exponent bytes: uint8, or torch's types for them
_MX_CODES = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())
_MX_SCALES = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())


def quantize_mxfp4(x: torch.Tensor, out=None):
    """float32 [rows, K] -> (codes uint8 [rows, K/2], scales uint8 [rows, 4 ceil(K/128)])."""
    x = _dev(x, "x", torch.float32)
    rows, k = x.shape
    dev = x.get_device()
    if out is None:
        codes = _new(rows, k // 2, torch.uint8, x.device)
        scales = _new(rows, 4 * _ceil128(k), torch.uint8, x.device)
    else:
        codes, scales = out
        _on(codes, "out codes", (rows, k // 2), _MX_CODES, dev)
        _on(scales, "out scales", (rows, 4 * _ceil128(k)), _MX_SCALES, dev)
    _launch(lib.mm_quantize_mxfp4, "mm_quantize_mxfp4", dev, x.data_ptr(), codes.data_ptr(), scales.data_ptr(),
            rows, k)
    return codes, scales


def _mx_pair(codes, scales, name: str, dev: int):
    """(rows, K) of MXFP4 codes [rows, K/2] with their scales, both on device dev."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise TypeError(f"{name} must be a 2-d GPU (HIP) tensor")
    rows, half = codes.shape
    _on(codes, name, (rows, half), _MX_CODES, dev)
    _on(scales, f"{name}_scale", (rows, 4 * _ceil128(2 * half)), _MX_SCALES, dev)
    return rows, 2 * half


def dequantize_mxfp4(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP4 codes [rows, K/2] and scales [rows, 4 ceil(K/128)] -> float32 [rows, K], exact."""
    _dev(codes, "codes")
    dev = codes.get_device()
    rows, k = _mx_pair(codes, scales, "codes", dev)
    if out is None:
        out = _new(rows, k, torch.float32, codes.device)
    else:
        _on(out, "out", (rows, k), _F32, dev)
    _launch(lib.mm_dequantize_mxfp4, "mm_dequantize_mxfp4", dev, codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
            rows, k)
    return out


@functools.lru_cache(maxsize=4096)
def mxfp4_workspace_size(m: int, n: int, k: int, src1_quantized: bool = False) -> int:
    return int(lib.mm_mul_mat_mxfp4_workspace_size(int(m), int(n), int(k), int(src1_quantized)))


def mul_mat_mxfp4_f32(w: torch.Tensor, w_scale: torch.Tensor, x: torch.Tensor, out=None, ws=None) -> torch.Tensor:
    """dst[M, N] = MXFP4(x)[M, K] . MXFP4(w)[N, K]^T; w codes [N, K/2] with scales [N, 4 ceil(K/128)]
    (quantize_mxfp4), x float32 [M, K], quantized within."""
    x = _dev(x, "x", torch.float32)
    m, k = x.shape
    dev = x.get_device()
    n, wk = _mx_pair(w, w_scale, "w", dev)
    if wk != k:
        raise ValueError(f"w has rows of {wk} values, x of {k}")
    out, ws, nbytes = _buffers(m, n, x.device, dev, out, mxfp4_workspace_size(m, n, k, False), ws)
    _launch(lib.mm_mul_mat_mxfp4_f32, "mm_mul_mat_mxfp4_f32", dev, w.data_ptr(), w_scale.data_ptr(), x.data_ptr(),
            out.data_ptr(), m, n, k, None if ws is None else ws.data_ptr(), nbytes)
    return out


def mul_mat_mxfp4_mxfp4(w: torch.Tensor, w_scale: torch.Tensor, a: torch.Tensor, a_scale: torch.Tensor,
                        out=None, ws=None) -> torch.Tensor:
    """mul_mat_mxfp4_f32 with src1 quantized already: a codes [M, K/2], a_scale [M, 4 ceil(K/128)]."""
    a = _dev(a, "a")
    dev = a.get_device()
    m, k = _mx_pair(a, a_scale, "a", dev)
    n, wk = _mx_pair(w, w_scale, "w", dev)
    if wk != k:
        raise ValueError(f"w has rows of {wk} values, a of {k}")
    out, ws, nbytes = _buffers(m, n, a.device, dev, out, mxfp4_workspace_size(m, n, k, True), ws)
    _launch(lib.mm_mul_mat_mxfp4_mxfp4, "mm_mul_mat_mxfp4_mxfp4", dev, w.data_ptr(), w_scale.data_ptr(), a.data_ptr(),
            a_scale.data_ptr(), out.data_ptr(), m, n, k, None if ws is None else ws.data_ptr(), nbytes)
    return out


def rms_norm_f32(x: torch.Tensor, weight=None, eps: float = 1e-5, residual=None, out_type: int = MM_TYPE_F32,
                 out=None, sum_out=None):
    """(y, v) with v = x + residual and y = v / sqrt(mean(v^2) + eps) * weight, float32 [T, D].

    y is float32, or (codes, scales) as quantize_f8(y) (out_type MM_TYPE_F8) or quantize_mxfp4(y)
    (MM_TYPE_MXFP4) gives them.  v is sum_out where given (x or residual itself: in place), else a new
    tensor; None without a residual and sum_out (v is x then)."""
    x = _dev(x, "x", torch.float32)
    t, d = x.shape
    dev = x.get_device()
    for name, v, shape in (("weight", weight, (d,)), ("residual", residual, (t, d)), ("sum_out", sum_out, (t, d))):
        if v is not None:
            _on(v, name, shape, _F32, dev)
    if sum_out is None and residual is not None:
        sum_out = _new(t, d, torch.float32, x.device)
    scales = None
    if out_type == MM_TYPE_F32:
        if out is None:
            out = _new(t, d, torch.float32, x.device)
        else:
            _on(out, "out", (t, d), _F32, dev)
        y, got = out, out
    else:
        f8 = out_type == MM_TYPE_F8
        if not f8 and out_type != MM_TYPE_MXFP4:
            raise ValueError("out_type must be MM_TYPE_F32, MM_TYPE_F8 or MM_TYPE_MXFP4")
        shape, sshape = ((t, d), (t, _ceil128(d))) if f8 else ((t, d // 2), (t, 4 * _ceil128(d)))
        if out is None:
            y = _new(*shape, torch.float8_e4m3fn if f8 else torch.uint8, x.device)
            scales = _new(*sshape, torch.float32 if f8 else torch.uint8, x.device)
        else:
            y, scales = out
            _on(y, "out codes", shape, _F8_DTYPES if f8 else _MX_CODES, dev)
            _on(scales, "out scales", sshape, _F32 if f8 else _MX_SCALES, dev)
        got = (y, scales)
    _launch(lib.mm_rms_norm_f32, "mm_rms_norm_f32", dev, x.data_ptr(), _ptr(residual), _ptr(weight), eps, _ptr(sum_out),
            out_type, y.data_ptr(), _ptr(scales), t, d)
    return got, sum_out


class _RouterStruct(ctypes.Structure):
    _fields_ = [("score", _int), ("top_k", _int), ("norm", _int), ("groups", _int), ("group_k", _int),
                ("group_top", _int), ("E", _i64), ("scale", ctypes.c_float), ("bias", _vp)]


_SCORES = {"softmax": 0, "sigmoid": 1}


class Router:
    """How tokens choose among e experts, for route_f32 (holds the bias tensor and the C struct).

    score: "softmax" or "sigmoid" of the logits; bias float32 [e] is added to the scores for the choice
    only.  groups > 1: experts in groups of e / groups neighbours, chosen from the group_k groups whose
    group_top (1 or 2) best sum highest.  norm: the chosen scores are divided by their sum; scale: then
    multiplied."""

    def __init__(self, e, top_k, score="softmax", bias=None, groups=1, group_k=1, group_top=1, norm=True, scale=1.0):
        if score not in _SCORES:
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        self.e, self.top_k, self.bias = int(e), int(top_k), bias
        if bias is not None:
            _on(_dev(bias, "bias"), "bias", (self.e,), _F32, bias.get_device())
        self.struct = _RouterStruct(_SCORES[score], self.top_k, int(bool(norm)), int(groups), int(group_k),
                                    int(group_top), self.e, float(scale), None)
        self._ref = ctypes.byref(self.struct)

    def _take(self, dev: int):
        if self.bias is not None:                      # where the tensor is now
            _on(self.bias, "bias", (self.e,), _F32, dev)
            self.struct.bias = self.bias.data_ptr()
        return self._ref


def route_f32(router: Router, logits: torch.Tensor, ids=None, weights=None):
    """(ids int32 [T, top_k], weights [T, top_k]) of logits float32 [T, e]; a slot without an expert
    (fewer than top_k to choose from) has id -1 and weight 0."""
    logits = _dev(logits, "logits", torch.float32)
    t, dev, k = logits.shape[0], logits.get_device(), router.top_k
    _on(logits, "logits", (t, router.e), _F32, dev)
    if ids is None:
        ids = _new(t, k, torch.int32, logits.device)
    else:
        _on(ids, "ids", (t, k), _I32, dev)
    if weights is None:
        weights = _new(t, k, torch.float32, logits.device)
    else:
        _on(weights, "weights", (t, k), _F32, dev)
    _launch(lib.mm_route_f32, "mm_route_f32", dev, router._take(dev), logits.data_ptr(), ids.data_ptr(),
            weights.data_ptr(), t)
    return ids, weights


class _MoeStruct(ctypes.Structure):
    _fields_ = [("type", _int), ("top_k", _int), ("norm", _int), ("D", _i64), ("F", _i64), ("E", _i64),
                ("router", _vp), ("gate", _vp), ("up", _vp), ("down", _vp),
                ("gate_scale", _vp), ("up_scale", _vp), ("down_scale", _vp)]


_MOE_POINTERS = ("router", "gate", "up", "down", "gate_scale", "up_scale", "down_scale")
_MOE_DTYPES = {MM_TYPE_Q4_0R: (torch.uint8,), MM_TYPE_F8: _F8_DTYPES, MM_TYPE_F16: (torch.float16,),
               MM_TYPE_MXFP4: _MX_CODES}


class MoeLayer:
    """The weights of a mixture-of-experts layer, for moe_f32 (holds the tensors and the C struct, whose
    addresses are the tensors' own at each call).

    router float32 [E, D]; gate, up (F x D per expert) and down (D x F) by mm_type:
    MM_TYPE_Q4_0R uint8 [E, repacked_bytes(rows, K)] (repack_q4_0 of each expert), MM_TYPE_F8
    e4m3 [E, rows, K] with float32 scales [E, ceil(rows/128), ceil(K/128)], MM_TYPE_F16 float16
    [E, rows, K], MM_TYPE_MXFP4 codes [E, rows, K/2] with scales [E, rows, 4 ceil(K/128)].  norm: the
    top_k probabilities are divided by their sum.

    router None: a layer for moe_routed_f32 only (router and norm play no part there); D then comes from
    gate, or for MM_TYPE_Q4_0R from d."""

    def __init__(self, mm_type, router, gate, up, down, f, top_k, gate_scale=None, up_scale=None,
                 down_scale=None, norm=True, d=None):
        if mm_type not in _MOE_DTYPES:
            raise ValueError("mm_type must be MM_TYPE_Q4_0R, MM_TYPE_F8, MM_TYPE_F16 or MM_TYPE_MXFP4")
        f, top_k = int(f), int(top_k)
        if router is not None:
            _dev(router, "router", torch.float32)
            e, width = router.shape
            at = router
        else:
            at = _dev(gate, "gate")
            if gate.dim() != (2 if mm_type == MM_TYPE_Q4_0R else 3):
                raise ValueError("gate must have its experts in the first of three dimensions (Q4_0R: of two)")
            e = gate.shape[0]
            if mm_type == MM_TYPE_Q4_0R:
                if d is None:
                    raise ValueError("d is needed for repacked experts without a router")
                width = int(d)
            else:
                width = gate.shape[2] * (2 if mm_type == MM_TYPE_MXFP4 else 1)
        if d is not None and int(d) != width:
            raise ValueError(f"d is {d}, the layer's tensors have {width}")
        d = width
        scales = (gate_scale, up_scale, down_scale) if mm_type in (MM_TYPE_F8, MM_TYPE_MXFP4) else (None,) * 3
        self.dev, self.device, self.d, self.f, self.e, self.top_k = at.get_device(), at.device, d, f, e, top_k
        self.tensors = (router, gate, up, down, *scales)
        self.struct = _MoeStruct(mm_type, top_k, int(bool(norm)), d, f, e)
        self._ref = ctypes.byref(self.struct)
        self._sizes, self._routed_sizes = {}, {}
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
            if router is not None:
                _on(router, "router", (e, d), _F32, dev)
            for name, w, scale, rows, k in zip(("gate", "up", "down"), rest[:3], rest[3:], (f, f, d), (d, d, f)):
                _on(w, name, (e, repacked_bytes(rows, k)) if kind == MM_TYPE_Q4_0R else
                    (e, rows, k // 2 if kind == MM_TYPE_MXFP4 else k), _MOE_DTYPES[kind], dev)
                if kind == MM_TYPE_F8:
                    _on(scale, f"{name}_scale", (e, _ceil128(rows), _ceil128(k)), _F32, dev)
                elif kind == MM_TYPE_MXFP4:
                    _on(scale, f"{name}_scale", (e, rows, 4 * _ceil128(k)), _MX_SCALES, dev)
            for field, t in zip(_MOE_POINTERS, self.tensors):
                setattr(self.struct, field, _ptr(t))
            self._seen = seen
        return self._ref

    def workspace_size(self, t: int) -> int:
        """Bytes of workspace for t tokens (0: t is out of range, or the layer's sizes are)."""
        if t not in self._sizes:
            self._sizes[t] = int(lib.mm_moe_workspace_size(self._ref, int(t)))
        return self._sizes[t]

    def routed_workspace_size(self, t: int) -> int:
        """workspace_size for moe_routed_f32."""
        if t not in self._routed_sizes:
            self._routed_sizes[t] = int(lib.mm_moe_routed_workspace_size(self._ref, int(t)))
        return self._routed_sizes[t]


_I32 = (torch.int32,)


def moe_f32(layer: MoeLayer, x: torch.Tensor, out=None, ids=None, weights=None, ws=None):
    """(dst [T, D], ids int32 [T, top_k], weights [T, top_k]) of the layer on x float32 [T, D]."""
    x = _dev(x, "x", torch.float32)
    if layer.tensors[0] is None:
        raise ValueError("the layer has no router: moe_routed_f32 takes it")
    t = x.shape[0]
    dev, k = layer.dev, layer.top_k
    _on(x, "x", (t, layer.d), _F32, dev)
    if ids is None:
        ids = _new(t, k, torch.int32, layer.device)
    else:
        _on(ids, "ids", (t, k), _I32, dev)
    if weights is None:
        weights = _new(t, k, torch.float32, layer.device)
    else:
        _on(weights, "weights", (t, k), _F32, dev)
    out, ws, nbytes = _buffers(t, layer.d, layer.device, dev, out, layer.workspace_size(t), ws)
    _launch(lib.mm_moe_f32, "mm_moe_f32", dev, layer._take(), x.data_ptr(), out.data_ptr(), ids.data_ptr(),
            weights.data_ptr(), t, None if ws is None else ws.data_ptr(), nbytes)
    return out, ids, weights


def moe_routed_f32(layer: MoeLayer, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, out=None, ws=None):
    """dst [T, D] of the layer's experts on x float32 [T, D] for a choice that is given: ids int32 and weights
    float32 [T, top_k] (route_f32); an id outside 0 .. E-1 is a slot without an expert."""
    x = _dev(x, "x", torch.float32)
    t = x.shape[0]
    dev, k = layer.dev, layer.top_k
    _on(x, "x", (t, layer.d), _F32, dev)
    _on(ids, "ids", (t, k), _I32, dev)
    _on(weights, "weights", (t, k), _F32, dev)
    out, ws, nbytes = _buffers(t, layer.d, layer.device, dev, out, layer.routed_workspace_size(t), ws)
    _launch(lib.mm_moe_routed_f32, "mm_moe_routed_f32", dev, layer._take(), x.data_ptr(), ids.data_ptr(),
            weights.data_ptr(), out.data_ptr(), t, None if ws is None else ws.data_ptr(), nbytes)
    return out


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
