"""CPU oracle of the AdamW step and of moments in 8 bits: TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; it shares no code with the HIP path.
float64 from the definition in include/moe.h.
"""
from __future__ import annotations

import numpy as np

__all__ = ["step", "decode", "encode", "E4M3"]

BLOCK = 128


def _values():
    """The 256 numbers of OCP E4M3 (bias 7, NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if c & 0x7F == 0x7F:
            v = np.nan
        out[c] = -v if c & 0x80 else v
    return out


E4M3 = _values()


def decode(codes, scale):
    """Values of codes uint8 [n] with scale bytes uint8 [ceil(n / 128)]."""
    codes = np.asarray(codes)
    s = 2.0 ** (np.asarray(scale, dtype=np.float64) - 127.0)
    return E4M3[codes] * np.repeat(s, BLOCK)[:len(codes)]


def encode(x, keep=False):
    """(codes, scale bytes) of values x: per block the smallest 2^e, -126 <= e <=
    126, with 448 2^e >= the largest finite magnitude; nearest code, ties to even;
    keep: what is above 0 gets the smallest code above 0 at least."""
    x = np.asarray(x, dtype=np.float64)
    n = len(x)
    codes = np.zeros(n, dtype=np.uint8)
    scale = np.zeros(-(-n // BLOCK), dtype=np.uint8)
    pos = E4M3[:127]
    for b in range(len(scale)):
        v = x[b * BLOCK:(b + 1) * BLOCK]
        fin = np.isfinite(v)
        amax = np.abs(v[fin]).max() if fin.any() else 0.0
        e = 0
        if amax > 0:
            e = int(np.clip(np.ceil(np.log2(amax / 448.0)), -126, 126))
            while e > -126 and 448.0 * 2.0 ** (e - 1) >= amax:
                e -= 1
            while e < 126 and 448.0 * 2.0 ** e < amax:
                e += 1
        scale[b] = e + 127
        for i, t in enumerate(v):
            if not np.isfinite(t):
                codes[b * BLOCK + i] = 0x7F
                continue
            y = min(abs(t) / 2.0 ** e, 448.0)
            d = np.abs(pos - y)
            c = int(np.argmin(d))
            if c + 1 < 127 and d[c + 1] == d[c] and (c & 1):
                c += 1
            if keep and t > 0 and c == 0:
                c = 1
            codes[b * BLOCK + i] = c | (0x80 if t < 0 and c else 0)
    return codes, scale


def step(w, g, m, v, *, lr, beta1, beta2, eps, weight_decay, t, grad_scale=1.0):
    """(w, m, v) float64 after one step."""
    g = np.asarray(g, dtype=np.float64) * grad_scale
    m = beta1 * np.asarray(m, dtype=np.float64) + (1.0 - beta1) * g
    v = beta2 * np.asarray(v, dtype=np.float64) + (1.0 - beta2) * g * g
    mh, vh = m / (1.0 - beta1 ** t), v / (1.0 - beta2 ** t)
    w = np.asarray(w, dtype=np.float64)
    return w - lr * (mh / (np.sqrt(vh) + eps) + weight_decay * w), m, v
