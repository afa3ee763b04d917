"""Polynomials that leave the formats' ranges (an iterate's element past 2, one
of b A + c A^2 past 65504): the matrix's result is not finite, never a finite
wrong one, and the other matrices of the stack are as they should be."""
import numpy as np
import pytest
import torch

from oracle import moe_ortho as oo
from tests import test_gpu_ortho as base
from tests.helpers import max_matrix_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B


@pytest.mark.parametrize("R,C", [(150, 150), (150, 300), (300, 150)])
@pytest.mark.parametrize("coeffs,steps", [((4.0, 0.0, 0.0), 4), ((1.0, 1e5, 0.0), 1), ((1.0, 0.0, 1e5), 1),
                                          ((1.0, 1.0, 1e5), 1)])
def test_past_the_range(B, R, C, coeffs, steps):
    print(f"case ortho overflow {R} {C} {coeffs} {steps}", flush=True)
    G = torch.randn((3, R, C), generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    G[1] = 0
    G[1, 20, 30] = 3.0
    G = G.bfloat16()
    s = B.make_ortho_shape(3, R, C, steps=steps, coeffs=coeffs)
    U = base._f64(B.orthogonalize(B.OrthoBuffers.allocate(s), G))
    assert not np.isfinite(U[1, 20, 30])
    rest = base._f64(G)[[0, 2]]
    assert max_matrix_err(U[[0, 2]], oo.orthogonalize(rest, steps, coeffs)) <= base.TOL
