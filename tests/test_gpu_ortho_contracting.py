"""Polynomials that shrink every singular value (a < 1), against the float64
oracle. Iterates are resolved to 2^-39, so each is off by at most 2^-40 an
element, which the later steps shrink a-fold each: 2^-40 a / (1 - a) in all,
beside the relative bound of test_gpu_ortho.py."""
import numpy as np
import pytest

from oracle import moe_ortho as oo
from tests import test_gpu_ortho as base

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B

CASES = [
    # (coeffs, steps)
    ((0.3, 0.0, 0.0), 16),
    ((0.3, -0.1, 0.05), 16),
    ((0.5, 0.0, 0.0), 32),
    ((0.5, -0.2, 0.05), 20),
    ((0.5, 0.0, 0.0), 8),       # the last that small matrices take on X X^T
    ((0.5, 0.0, 0.0), 9),
    ((0.9, -0.3, 0.1), 32),
]


@pytest.mark.parametrize("E,R,C,dtype", [(3, 24, 40, "bf16"), (2, 128, 90, "f32"), (2, 140, 150, "bf16")])
@pytest.mark.parametrize("coeffs,steps", CASES)
def test_contracting_polynomials(B, E, R, C, dtype, coeffs, steps):
    print(f"case ortho contracting E={E} R={R} C={C} {dtype} {coeffs} {steps}", flush=True)
    G = base._grad(E, R, C, dtype, 7)
    s = B.make_ortho_shape(E, R, C, steps=steps, grad=dtype, coeffs=coeffs)
    U = B.orthogonalize(B.OrthoBuffers.allocate(s), G)
    want = oo.orthogonalize(base._f64(G), steps, tuple(float(np.float32(c)) for c in coeffs))
    got, a = base._f64(U), coeffs[0]
    assert np.isfinite(got).all()
    for e in range(E):
        bound = base.TOL * np.linalg.norm(want[e]) + 2.0 ** -40 * a / (1 - a) * np.sqrt(R * C)
        assert np.linalg.norm(got[e] - want[e]) <= bound
