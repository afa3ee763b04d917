"""CPU oracle of the dense products with bias, activation and residual: TEST
INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the HIP path.
float64 on the exact bf16 / fp32 inputs, from the definition in include/moe.h.
"""
from __future__ import annotations

import numpy as np

__all__ = ["activate", "slope_times", "linear", "linear_backward"]

A, B = np.sqrt(2.0 / np.pi), 0.044715


def _sigmoid(x):
    q = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, q) / (1.0 + q)


def activate(P, act: str):
    if act == "relu":
        return np.maximum(P, 0.0)
    if act == "silu":
        return P * _sigmoid(P)
    if act == "gelu":
        return 0.5 * P * (1.0 + np.tanh(A * (P + B * P ** 3)))
    if act == "swiglu":
        g, u = np.split(P, 2, axis=1)
        return g * _sigmoid(g) * u
    return P


def slope_times(dY, P, act: str):
    """dL/dP given dL/d activate(P)."""
    if act == "none":
        return dY
    if act == "relu":
        return np.where(P > 0, dY, 0.0)
    if act == "gelu":
        th = np.tanh(A * (P + B * P ** 3))
        return dY * (0.5 * (1.0 + th) + 0.5 * P * (1.0 - th ** 2) * A * (1.0 + 3.0 * B * P ** 2))
    if act == "silu":
        s = _sigmoid(P)
        return dY * (s + P * s * (1.0 - s))
    g, u = np.split(P, 2, axis=1)
    s = _sigmoid(g)
    return np.concatenate([dY * u * (s + g * s * (1.0 - s)), dY * g * s], axis=1)


def linear(X, W, bias=None, residual=None, act="none"):
    """(Y, P) float64."""
    P = X @ W.T
    if bias is not None:
        P = P + bias
    Y = activate(P, act)
    return (Y if residual is None else Y + residual), P


def linear_backward(dY, X, W, P, act="none"):
    """(dX, dW, dbias, dP) float64; P as it was kept."""
    dP = slope_times(dY, P, act)
    return dP @ W, dP.T @ X, dP.sum(0), dP
