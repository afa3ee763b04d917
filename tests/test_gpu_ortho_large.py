"""Single matrices up to the largest sides, whose every element is known: with
one entry in each row and column (a scaled permutation) a matrix's singular
values are its entries' magnitudes, and the polynomial acts on each entry alone.
Bound as in test_gpu_ortho.py; everything else must be zero."""
import pytest
import torch

from oracle import moe_ortho as oo
from tests import test_gpu_ortho as base

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B


@pytest.mark.parametrize("R,C", [(16384, 16384), (9001, 16384), (16384, 12345), (16383, 200), (16384, 4096)])
def test_scaled_permutations(B, R, C):
    print(f"case ortho large {R} x {C}", flush=True)
    m = min(R, C)
    g = torch.Generator(device=DEV).manual_seed(R + C)
    rows = torch.randperm(R, generator=g, device=DEV)[:m]
    cols = torch.randperm(C, generator=g, device=DEV)[:m]
    val = torch.randn(m, generator=g, device=DEV).bfloat16()
    G = torch.zeros((1, R, C), dtype=torch.bfloat16, device=DEV)
    G[0, rows, cols] = val
    U = B.orthogonalize(B.OrthoBuffers.allocate(B.make_ortho_shape(1, R, C)), G)
    torch.cuda.synchronize()
    s = val.double()
    s = s / (s.norm() + 1e-7)
    a, b, c = oo.COEFFS
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    got = U[0, rows, cols].double()
    assert torch.isfinite(got).all()
    assert ((got - s).norm() / s.norm()).item() <= base.TOL
    U[0, rows, cols] = 0
    assert not U.any().item()
