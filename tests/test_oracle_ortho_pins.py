"""CPU pins of the orthogonalisation oracle: the polynomial acts on singular
values alone, and closed forms."""
import numpy as np
import pytest

from oracle import moe_ortho as oo


def _poly(s, steps, coeffs):
    a, b, c = coeffs
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return s


@pytest.mark.parametrize("R,C", [(5, 9), (9, 5), (7, 7), (1, 4), (4, 1), (1, 1)])
@pytest.mark.parametrize("steps,coeffs", [(5, oo.COEFFS), (1, oo.COEFFS), (12, (1.5, -0.5, 0.0))])
def test_moves_singular_values_only(R, C, steps, coeffs):
    G = np.random.default_rng(R * 10 + C).normal(size=(2, R, C))
    got = oo.orthogonalize(G, steps, coeffs, eps=1e-3)
    for e in range(2):
        u, s, vt = np.linalg.svd(G[e], full_matrices=False)
        want = (u * _poly(s / (np.linalg.norm(G[e]) + 1e-3), steps, coeffs)) @ vt
        np.testing.assert_allclose(got[e], want, rtol=0, atol=1e-11)


def test_cubic_converges_to_the_orthogonal_factor():
    G = np.random.default_rng(3).normal(size=(1, 6, 11))
    u, _, vt = np.linalg.svd(G[0], full_matrices=False)
    np.testing.assert_allclose(oo.orthogonalize(G, 40, (1.5, -0.5, 0.0), 0.0)[0], u @ vt, atol=1e-12)


def test_zero_and_nonfinite_matrices():
    G = np.random.default_rng(4).normal(size=(4, 3, 5))
    G[1] = 0.0
    G[2, 1, 1] = np.inf
    U = oo.orthogonalize(G)
    assert not U[1].any() and np.all(np.isnan(U[2]))
    np.testing.assert_array_equal(U[[0, 3]], oo.orthogonalize(G[[0, 3]]))


def test_muon_step_by_hand():
    """Rank one, cubic with one step: U = (1.5 - 0.5) u v^T."""
    g = np.array([[[3.0, 4.0]]])
    m, W = oo.muon_step(g, np.array([[[2.0, 0.0]]]), np.ones((1, 1, 2)), 0.1, 0.5, 0.2, 2.0, False,
                        steps=1, coeffs=(1.5, -0.5, 0.0), eps=0.0)
    np.testing.assert_allclose(m, [[[4.0, 4.0]]])
    np.testing.assert_allclose(W, 0.98 - 0.2 / np.sqrt(2) * np.ones((1, 1, 2)))
    m, W = oo.muon_step(g, np.array([[[2.0, 0.0]]]), np.ones((1, 1, 2)), 0.1, 0.5, 0.0, 1.0, True,
                        steps=1, coeffs=(1.5, -0.5, 0.0), eps=0.0)
    np.testing.assert_allclose(W, 1.0 - 0.1 * np.array([[[5.0, 6.0]]]) / np.sqrt(61.0))
