"""CPU oracle of the routing balance: TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the HIP path.
Everything is float64 on the exact fp32 logits, sequence by sequence.

With p = softmax over a token's E logits, lse its log-sum-exp, and the live
tokens of a sequence those inside its bounds whose mask is set:

* balance = mean over the sequences with live tokens of
  E * sum_e (share of the live (token, slot) pairs routed to e) * (mean p_e);
* z = mean over all live tokens of lse^2.

A logit of -inf is an expert that is off; a row of them alone has p = 0 and
gives nothing to z, but is live.
"""
from __future__ import annotations

import numpy as np

__all__ = ["balance", "balance_backward"]


def _rows(logits):
    """p [T, E] and lse [T]; rows of -inf alone give p = 0 and lse = 0."""
    z = np.asarray(logits, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        top = np.max(z, axis=1, keepdims=True) if z.size else np.zeros((z.shape[0], 1))
        off = np.isneginf(top)
        e = np.exp(z - np.where(off, 0.0, top))
        s = np.sum(e, axis=1, keepdims=True)
        p = np.where(off, 0.0, e / np.where(off, 1.0, s))
        lse = np.where(off, 0.0, top + np.log(np.where(off, 1.0, s)))[:, 0]
    return p, lse


def _members(T, seq_offsets, mask):
    """The live tokens of each sequence."""
    bounds = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    live = np.ones(T, dtype=bool) if mask is None else np.asarray(mask) != 0
    out = []
    for q in range(len(bounds) - 1):
        t = np.arange(bounds[q], max(bounds[q], bounds[q + 1]))
        out.append(t[live[t]])
    return out


def balance(logits, topk_idx, seq_offsets=None, mask=None):
    """dict of loss [2], counts [E], seq_counts [S, E], seq_probs [S, E], seq_scale [S + 1]."""
    p, lse = _rows(logits)
    idx = np.asarray(topk_idx, dtype=np.int64)
    T, E = p.shape
    k = idx.shape[1]
    members = _members(T, seq_offsets, mask)
    S = len(members)
    used = sum(len(m) > 0 for m in members)
    total = sum(len(m) for m in members)
    counts = np.zeros((S, E), dtype=np.int64)
    probs = np.zeros((S, E))
    scale = np.zeros(S + 1)
    loss = np.zeros(2)
    for q, m in enumerate(members):
        if len(m) == 0:
            continue
        pairs = idx[m].reshape(-1)
        counts[q] = np.bincount(pairs[(pairs >= 0) & (pairs < E)], minlength=E)
        probs[q] = p[m].mean(axis=0)
        share = counts[q] / (k * len(m))
        loss[0] += E * np.sum(share * probs[q]) / used
        loss[1] += np.sum(lse[m] ** 2) / total
        scale[q] = E / (used * k * len(m) ** 2)
    if total:
        scale[S] = 1.0 / total
    return {"loss": loss, "counts": counts.sum(axis=0), "seq_counts": counts, "seq_probs": probs, "seq_scale": scale}


def balance_backward(logits, topk_idx, topk_w, d_topk_w, renorm, d_loss, seq_offsets=None, mask=None):
    """d_logits [T, E] of d_loss . loss and, unless d_topk_w is None, of the
    routing weights: renormalised w (dw - <w, dw>) on the selected experts,
    otherwise p (G - <p, G>) with G = dw placed on them (summed where an
    expert is named twice)."""
    p, lse = _rows(logits)
    idx = np.asarray(topk_idx, dtype=np.int64)
    f = balance(logits, topk_idx, seq_offsets, mask)
    d = np.zeros_like(p)
    T = p.shape[0]
    for q, m in enumerate(_members(T, seq_offsets, mask)):
        v = d_loss[0] * f["seq_scale"][q] * f["seq_counts"][q]
        d[m] += p[m] * (v - (p[m] @ v)[:, None])
        d[m] += 2.0 * d_loss[1] * f["seq_scale"][-1] * lse[m][:, None] * p[m]
    if d_topk_w is not None:
        dw = np.asarray(d_topk_w, dtype=np.float64)
        G = np.zeros_like(p)
        t = np.repeat(np.arange(T), idx.shape[1])
        if renorm:
            w = np.asarray(topk_w, dtype=np.float64)
            np.add.at(d, (t, idx.reshape(-1)), (w * (dw - np.sum(w * dw, axis=1, keepdims=True))).reshape(-1))
        else:
            np.add.at(G, (t, idx.reshape(-1)), dw.reshape(-1))
            d += p * (G - np.sum(p * G, axis=1, keepdims=True))
    return d
