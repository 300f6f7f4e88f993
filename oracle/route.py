"""Routing to experts in float64: scores, choice by score plus bias within the best groups, the chosen scores as weights."""
from __future__ import annotations

import numpy as np


def route(logits, top_k, score="softmax", bias=None, groups=1, group_k=1, group_top=1, norm=True, scale=1.0):
    """(ids int32 [T, top_k], weights float64): -1 and 0 in slots without an expert, NaN weights where a logit is NaN (or
    infinite under a softmax)."""
    t, e = logits.shape
    b = np.zeros(e) if bias is None else bias.astype(np.float64)
    ids, weights = np.full((t, top_k), -1, np.int32), np.zeros((t, top_k))
    with np.errstate(all="ignore"):
        for i in range(t):
            l = logits[i].astype(np.float64)
            if score == "softmax":
                top = np.nanmax(l) if not np.isnan(l).all() else np.nan
                s = np.where(l == -np.inf, 0.0, np.exp(l - top))
                s = s / s.sum() if s.sum() > 0 else s
            else:
                s = 1 / (1 + np.exp(-l))
            c = s + b
            free = (l != -np.inf) & (b != -np.inf)
            if groups > 1 and group_k < groups:
                per = e // groups
                worth = np.full(groups, -np.inf)
                for g in range(groups):
                    m = np.sort([c[j] for j in range(g * per, (g + 1) * per) if free[j] and not np.isnan(c[j])])[::-1]
                    if len(m):
                        worth[g] = m[:group_top].sum()
                best = np.argsort(-worth, kind="stable")[:group_k]
                free &= np.isin(np.arange(e) // per, best)
            order = sorted(np.flatnonzero(free), key=lambda j: (np.isnan(c[j]), -c[j] if not np.isnan(c[j]) else 0, j))
            take = order[:top_k]
            ids[i, :len(take)] = take
            w = s[take]
            if norm:
                w = w / w.sum() if w.sum() > 0 else w * 0
            weights[i, :len(take)] = w * scale
            if np.isnan(l).any() or (score == "softmax" and (l == np.inf).any()):
                weights[i] = np.nan
    return ids, weights
