"""CPU pins of the routing-balance oracle: closed forms, per-token loops and
finite differences."""
import math

import numpy as np
import pytest

from oracle import moe_balance as ob


def _case(T, E, k, seed, S=1, drop=0.0):
    g = np.random.default_rng(seed)
    z = g.normal(size=(T, E))
    idx = np.argsort(-z, axis=1)[:, :k]
    off = np.concatenate([[0], np.sort(g.integers(0, T + 1, size=S - 1)), [T - (T // 7 if S > 1 else 0)]])
    off[-1] = max(off[-1], off[-2])
    mask = (g.random(T) >= drop).astype(np.uint8)
    return z, idx, off, mask


def test_uniform_routing_has_loss_one():
    T, E, k = 12, 6, 2
    idx = np.stack([np.arange(T) % E, (np.arange(T) + 3) % E], 1)
    f = ob.balance(np.zeros((T, E)), idx)
    assert f["loss"][0] == pytest.approx(1.0)
    assert f["loss"][1] == pytest.approx(math.log(E) ** 2)
    assert np.array_equal(f["counts"], np.full(E, T * k // E))


def test_collapsed_routing_has_loss_E():
    E = 8
    z = np.full((5, E), -math.inf)
    z[:, 2] = 1.5
    f = ob.balance(z, np.full((5, 1), 2))
    assert f["loss"][0] == pytest.approx(E)
    assert f["loss"][1] == pytest.approx(1.5 ** 2)


def test_matches_token_loops():
    z, idx, off, mask = _case(40, 7, 3, 1, S=5, drop=0.3)
    f = ob.balance(z, idx, off, mask)
    S, E, k = 5, 7, 3
    loss, used, zs, n = 0.0, 0, 0.0, 0
    for q in range(S):
        c, P, live = [0] * E, [0.0] * E, 0
        for t in range(off[q], off[q + 1]):
            if not mask[t]:
                continue
            live += 1
            den = sum(math.exp(v) for v in z[t])
            for e in range(E):
                P[e] += math.exp(z[t][e]) / den
            for j in range(k):
                c[idx[t][j]] += 1
            zs += math.log(den) ** 2
        assert list(f["seq_counts"][q]) == c
        n += live
        if live:
            used += 1
            loss += E * sum(c[e] / (k * live) * P[e] / live for e in range(E))
    assert f["loss"][0] == pytest.approx(loss / used, rel=1e-12)
    assert f["loss"][1] == pytest.approx(zs / n, rel=1e-12)


def test_dead_batch_is_zero():
    z, idx, _, _ = _case(9, 4, 2, 2)
    f = ob.balance(z, idx, [0, 9], np.zeros(9))
    assert not f["loss"].any() and not f["counts"].any() and not f["seq_scale"].any()
    assert not ob.balance_backward(z, idx, None, None, True, (1.0, 1.0), [0, 9], np.zeros(9)).any()


def _route_weights(z, idx, renorm):
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, idx, 1)
    return w / w.sum(1, keepdims=True) if renorm else w


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("S,drop", [(1, 0.0), (4, 0.3)])
def test_gradient_matches_differences(renorm, S, drop):
    z, idx, off, mask = _case(23, 6, 2, 3 + S, S=S, drop=drop)
    dw = np.random.default_rng(9).normal(size=idx.shape)
    gl = (0.7, 0.3)
    counts = ob.balance(z, idx, off, mask)["counts"].copy()

    def total(zz):
        f = ob.balance(zz, idx, off, mask)
        assert np.array_equal(f["counts"], counts)
        return gl[0] * f["loss"][0] + gl[1] * f["loss"][1] + np.sum(dw * _route_weights(zz, idx, renorm))

    d = ob.balance_backward(z, idx, _route_weights(z, idx, renorm), dw, renorm, gl, off, mask)
    g = np.random.default_rng(5)
    for _ in range(12):
        v = g.normal(size=z.shape)
        h = 1e-5
        num = (total(z + h * v) - total(z - h * v)) / (2 * h)
        assert num == pytest.approx(np.sum(d * v), rel=1e-6, abs=1e-9)


def test_dead_rows_and_experts_that_are_off():
    """A row of -inf alone adds nothing and gets nothing; an expert that is
    off gets a zero gradient."""
    z, idx, _, _ = _case(10, 5, 2, 7)
    z[3] = -math.inf
    z[:, 4] = -math.inf
    f = ob.balance(z, idx)
    d = ob.balance_backward(z, idx, None, None, True, (1.0, 1.0))
    assert np.all(np.isfinite(f["loss"])) and np.all(np.isfinite(d))
    assert not d[3].any() and not d[:, 4].any()
    assert f["seq_probs"][0].sum() == pytest.approx(9 / 10)
