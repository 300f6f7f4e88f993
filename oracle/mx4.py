"""MXFP4 (OCP microscaling, e2m1 with one power of two per 32 values): quantizer, decode and product, in NumPy.

Values: code = sign, 2 exponent bits (bias 1), 1 fraction bit; a scale byte b is 2^(b - 127), 255 is NaN.  Packed: element
2 i of a row in the low half of its byte i; a row's scale bytes are padded with 127 to whole 4 bytes.

Quantizer: byte = max(floor(log2(amax)) - 2 + 127, 0), code = the e2m1 value nearest to x / 2^(byte - 127), ties to the
even code, magnitudes over 6 become 6; a block that holds an infinity or NaN has byte 255 and codes 0.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
POS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
VALUES = np.concatenate([POS, -POS])
MID = (POS[1:] + POS[:-1]) / 2


def encode(v):
    """float64 -> e2m1 codes, ties to even, saturating; the sign bit is the value's."""
    a = np.abs(v)
    lo = np.searchsorted(MID, a, side="left")                # first midpoint >= a: code lo, or a tie
    tie = (lo < len(MID)) & (a == MID[np.minimum(lo, len(MID) - 1)])
    code = lo + np.where(tie & (lo % 2 == 1), 1, 0)
    return (code | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def padded(k):
    return 4 * -(-k // 128)


def quantize(x):
    """float32 [rows, K] -> (codes uint8 [rows, K/2], scales uint8 [rows, padded(K)])."""
    x = np.asarray(x, dtype=np.float32)
    n, k = x.shape
    b = x.reshape(n, k // BLOCK, BLOCK).astype(np.float64)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(axis=2)
    e = np.frexp(amax)[1] - 1                                # floor(log2), exact
    e = np.maximum(np.where(amax > 0, e - 2, -127), -127)
    codes = encode(np.ldexp(b, -e[..., None])).reshape(n, k)
    codes = np.where(np.repeat(bad, BLOCK, axis=1), 0, codes).astype(np.uint8)
    scales = np.full((n, padded(k)), 127, np.uint8)
    scales[:, :k // BLOCK] = np.where(bad, 255, e + 127)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales


def dequantize(codes, scales):
    n, half = codes.shape
    c = np.empty((n, 2 * half), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    e = np.repeat(scales[:, :2 * half // BLOCK].astype(np.int64), BLOCK, axis=1)
    return np.where(e == 255, np.nan, np.ldexp(VALUES[c], e - 127))


def mul_mat(w, ws, a, a_s):
    """dst[M, N] and the sum of the magnitudes of its terms, float64."""
    wv, av = dequantize(w, ws), dequantize(a, a_s)
    return av @ wv.T, np.abs(av) @ np.abs(wv).T
