"""Scratch sizes never fall as a stack or a batch grows: a scratch allocated for
the largest serves every smaller one."""
import os

import pytest

from tests.helpers import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


@pytest.fixture(scope="module")
def B():
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


# X X^T in parts up to 64 tiles: 21, 6, 3, 1 and no matrices; a shape without parts; a small side
SHAPES = [(256, 2048), (2048, 256), (130, 16384), (334, 3542), (640, 2048), (1024, 4096), (1500, 1600), (1536, 4096),
          (300, 1000), (128, 4096), (24, 33)]


@pytest.mark.parametrize("R,C", SHAPES)
def test_ortho_scratch_grows_with_the_stack(B, R, C):
    sizes = [B.moe_ortho_workspace_size(B.make_ortho_shape(E, R, C)) for E in range(1, 200)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [E + 1 for E in range(198) if sizes[E] > sizes[E + 1]]
    assert B.moe_ortho_workspace_size(B.make_ortho_shape(10 ** 4, R, C)) >= sizes[-1]
    assert B.moe_ortho_workspace_size(B.make_ortho_shape(0, R, C)) <= sizes[0]
