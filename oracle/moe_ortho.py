"""CPU oracle of the Newton-Schulz orthogonalisation: TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the HIP path.
Everything is float64 on the exact input values, one matrix at a time, from the
definition: X = G / (|G|_F + eps), then X <- a X + (b A + c A A) X with
A = X X^T (or, for more rows than columns, the same on the right).
"""
from __future__ import annotations

import numpy as np

__all__ = ["orthogonalize", "muon_step", "COEFFS"]

COEFFS = (3.4445, -4.7750, 2.0315)


def orthogonalize(G, steps: int = 5, coeffs=COEFFS, eps: float = 1e-7):
    """float64 [E, R, C]; a matrix with a NaN or an infinity gives NaN throughout."""
    a, b, c = coeffs
    G = np.asarray(G, dtype=np.float64)
    out = np.zeros_like(G)
    for e in range(G.shape[0]):
        g = G[e]
        if not np.all(np.isfinite(g)):
            out[e] = np.nan
            continue
        norm = np.sqrt(np.sum(g * g))
        if norm == 0.0:
            continue
        X = g / (norm + eps)
        for _ in range(steps):
            if X.shape[0] <= X.shape[1]:
                A = X @ X.T
                X = a * X + (b * A + c * (A @ A)) @ X
            else:
                A = X.T @ X
                X = a * X + X @ (b * A + c * (A @ A))
        out[e] = X
    return out


def muon_step(grad, momentum, W, lr, mu, weight_decay, scale, nesterov, **kw):
    """The new (momentum, W) of one optimizer step."""
    g = np.asarray(grad, dtype=np.float64)
    m = mu * np.asarray(momentum, dtype=np.float64) + g
    u = g + mu * m if nesterov else m
    W = np.asarray(W, dtype=np.float64) * (1.0 - lr * weight_decay) - lr * scale * orthogonalize(u, **kw)
    return m, W
