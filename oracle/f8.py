"""e4m3 with one fp32 scale per block of 128: quantizer, decode and product, in NumPy.

Values: byte = sign, 4 exponent bits (bias 7), 3 fraction bits; exponent field 0 is subnormal
(fraction * 2^-9); 0x7f and 0xff are NaN; the largest value is 448.  Blocks are 1 x 128 (activations)
or 128 x 128 (weights) and may be short at the end of a row and of the rows.

Quantizer, one correctly rounded fp32 operation each: d = max(amax / 448, 2^-126), id = 1 / d,
v = x * id; code = the e4m3 value nearest to v, ties to the even code.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _table():
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = np.nan if b & 0x7f == 0x7f else -x if b & 0x80 else x
    return v


VALUES = _table()
_POS = VALUES[:0x7f]                                     # ascending: codes 0 .. 0x7e
_MID = (_POS[1:] + _POS[:-1]) / 2                        # exact in float64


def encode(v):
    """float32 values of magnitude at most 464 -> nearest e4m3 codes, ties to even; NaN -> 0x7f."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    lo = np.searchsorted(_MID, a, side="left")           # first midpoint >= a: code lo, or a tie
    tie = (lo < len(_MID)) & (a == _MID[np.minimum(lo, len(_MID) - 1)])
    code = lo + np.where(tie & (lo % 2 == 1), 1, 0)
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7f, code).astype(np.uint8)


def quantize(x, block_rows):
    """float32 [rows, K] -> (codes uint8 [rows, K], scales float32 [ceil(rows/R), ceil(K/128)])."""
    x = np.asarray(x, dtype=np.float32)
    n, k = x.shape
    nb, kb = -(-n // block_rows), -(-k // BLOCK)
    codes = np.empty((n, k), np.uint8)
    scales = np.empty((nb, kb), np.float32)
    with np.errstate(all="ignore"):
        for i in range(nb):
            for j in range(kb):
                at = np.s_[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
                blk = x[at]
                amax = np.float32(np.nanmax(np.abs(blk))) if not np.isnan(blk).all() else np.float32(0)
                d = np.maximum(np.float32(amax / np.float32(448)), np.float32(2.0 ** -126))
                scales[i, j] = d
                codes[at] = encode(blk * np.float32(np.float32(1) / d))
    return codes, scales


def dequantize(codes, scales, block_rows):
    n, k = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), block_rows, 0)[:n], BLOCK, 1)[:, :k]
    with np.errstate(invalid="ignore"):
        return VALUES[codes] * s


def mul_mat(w, ws, a, a_s):
    """dst[M, N] and the sum of the magnitudes of its terms, float64."""
    wv, av = dequantize(w, ws, BLOCK), dequantize(a, a_s, 1)
    return av @ wv.T, np.abs(av) @ np.abs(wv).T
