"""CPU oracle of the choice of experts by scores, bias and groups: TEST
INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the HIP path.
Everything is float64 on the exact fp32 inputs, one token at a time, from the
definition in include/moe.h (the pages keep the router outside the layer).
"""
from __future__ import annotations

import numpy as np

__all__ = ["scores", "choose", "choose_backward"]


def _sigmoid(x):
    q = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, q) / (1.0 + q)


def scores(z, score: str):
    """s[e] of one token; 0 where the logit is -inf."""
    z = np.asarray(z, dtype=np.float64)
    live = z > -np.inf
    s = np.zeros_like(z)
    if not live.any():
        return s
    if score == "sigmoid":
        s[live] = _sigmoid(z[live])
    else:
        e = np.exp(z[live] - z[live].max())
        s[live] = e / e.sum()
    return s


def _weights(z, ids, score, renorm):
    """s (or s over the sum of the chosen, from logits moved by a common shift)."""
    if not renorm:
        return scores(z, score)[ids]
    x = np.asarray(z, dtype=np.float64)[ids]
    if score == "softmax":
        a = np.exp(x - x.max())
    else:   # sigmoid(x) / e^min(max x, 0)
        ref = min(x.max(), 0.0)
        a = np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))),
                     np.exp(np.minimum(x - ref, 0.0)) / (1.0 + np.exp(-np.abs(x))))
    return a / a.sum()


def choose(logits, k, score="softmax", renorm=True, bias=None, groups=1, kept=None, top=1, scale=1.0, mask=None):
    """topk_idx int64 [T, k] (-1: none left), topk_w float64 [T, k]."""
    Z = np.asarray(logits, dtype=np.float64)
    T, E = Z.shape
    kept = groups if kept is None else kept
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    idx = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        z = Z[t]
        if mask is not None and not mask[t]:
            continue
        if np.isnan(z).any() or (z == np.inf).any() or np.isnan(b).any() or (b == np.inf).any():
            idx[t], w[t] = np.arange(k), np.nan
            continue
        live = (z > -np.inf) & (b > -np.inf)
        s = scores(z, score)
        c = z if bias is None else s + np.where(np.isinf(b), 0.0, b)
        by = s if bias is None and top == 2 else c
        allowed = live.copy()
        if groups > 1:
            n = E // groups
            value = []
            for g in range(groups):
                ids = [e for e in range(g * n, (g + 1) * n) if live[e]]
                best = sorted((by[e] for e in ids), reverse=True)[:top]
                value.append((-sum(best), g) if best else (np.inf, g))
            chosen = [g for v, g in sorted(value)[:kept]]
            allowed &= np.isin(np.arange(E) // n, chosen)
        ids = sorted(np.flatnonzero(allowed), key=lambda e: (-c[e], e))[:k]
        if ids:
            idx[t, :len(ids)] = ids
            w[t, :len(ids)] = scale * _weights(z, ids, score, renorm)
    return idx, w


def choose_backward(logits, topk_idx, d_topk_w, score="softmax", renorm=True, scale=1.0):
    """d_logits float64 [T, E]; ids outside [0, E) pass nothing."""
    Z = np.asarray(logits, dtype=np.float64)
    T, E = Z.shape
    d = np.zeros_like(Z)
    for t in range(T):
        slots = [j for j, e in enumerate(topk_idx[t]) if 0 <= e < E]
        ids = np.array([topk_idx[t][j] for j in slots], dtype=np.int64)
        dw = scale * np.array([d_topk_w[t][j] for j in slots], dtype=np.float64)
        if len(ids) == 0:
            continue
        if score == "softmax" and not renorm:
            G = np.zeros(E)
            np.add.at(G, ids, dw)
            p = scores(Z[t], score)
            d[t] = p * (G - p @ G)
            continue
        x = Z[t][ids]
        if renorm:
            p = _weights(Z[t], ids, score, True)
            v = p * (dw - p @ dw)
        else:
            v = scores(Z[t], score)[ids] * dw
        if score == "sigmoid":
            v = v * _sigmoid(-x)
        np.add.at(d[t], ids, v)
    return d
