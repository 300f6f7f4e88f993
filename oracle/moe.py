"""Mixture-of-experts layer in float64, with a bound of an fp32 evaluation's error.

logits = x . router^T; p = softmax; the top_k experts of a token by logit, ties to the lower index;
weights p, or p over the sum of the chosen; h = silu(gate x) * (up x); dst = sum of weights * down h.
"""
from __future__ import annotations

import numpy as np


def select(x, router, top_k, norm):
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    z = np.exp(logits - logits.max(axis=1, keepdims=True))
    p = z / z.sum(axis=1, keepdims=True)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, ids, 1)
    return ids.astype(np.int32), (w / w.sum(axis=1, keepdims=True) if norm else w)


def act_error(v):
    """Bound of |error| per element of v [..., K] where activations are held in blocks of 32 as two binary16 numbers,
    scaled by a power of two that puts the block's largest magnitude in [2^14, 2^15).

    Of a scaled value in [2^e, 2^(e+1)) the first keeps 11 bits, off by at most 2^(e-11); the second keeps 11 bits of that,
    off by at most 2^(e-23), or half of binary16's smallest step, 2^-25, where that is more (e < -2).  So the error is at
    most 2^-23 of the value, or 2^-39 of the block's largest (2^-25 of at least 2^14)."""
    a = np.abs(v)
    k = a.shape[-1]
    top = np.maximum.reduceat(a, np.arange(0, k, 32), axis=-1).repeat(32, axis=-1)[..., :k]
    return np.maximum(2.0 ** -23 * a, 2.0 ** -39 * top)


def layer(x, router, gate, up, down, top_k, norm, act_eps, sum_eps):
    """dst, ids, weights and a bound of |dst - exact| where activations enter products with an error of act_eps relative
    and act_error, and a product's sum is off by at most sum_eps times the sum of its terms' magnitudes.
    gate, up [E, F, D] and down [E, D, F] as float64 values."""
    x = x.astype(np.float64)
    ids, w = select(x, router, top_k, norm)
    dst, err = np.zeros_like(x), np.zeros_like(x)
    c = act_eps + sum_eps
    for t in range(x.shape[0]):
        for j in range(top_k):
            e = ids[t, j]
            g, u = gate[e] @ x[t], up[e] @ x[t]
            ex = c * np.abs(x[t]) + act_error(x[t])
            eg, eu = np.abs(gate[e]) @ ex, np.abs(up[e]) @ ex
            s = g / (1 + np.exp(-g))
            h = s * u
            # |silu'| <= 1.1; the elementwise part itself within 8 fp32 roundings
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * 2.0 ** -24 * np.abs(h)
            y = down[e] @ h
            dst[t] += w[t, j] * y
            # weights within 16 fp32 roundings
            held = c * (np.abs(h) + eh) + act_error(np.abs(h) + eh)
            err[t] += w[t, j] * (np.abs(down[e]) @ (eh + held) + 2.0 ** -20 * np.abs(y))
    return dst, ids, w, err
