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


@pytest.mark.parametrize("E", [8, 128, 256, 257, 512, 513, 1024])
@pytest.mark.parametrize("S", [1, 48])
def test_balance_scratch_grows_with_the_batch(B, E, S):
    T = sorted({t + d for c in (16, 32, 64, 96, 128, 256, 1024) for t in (8 * c, 1023 * c, 1024 * c, 2048 * c)
                for d in (-1, 0, 1, 7)})
    sizes = [B.moe_balance_scratch_bytes(B.make_shape(t, 256, 128, E, 2), S) for t in T]
    assert all(n > 0 for n in sizes)
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [T[i] for i in range(len(T) - 1) if sizes[i] > sizes[i + 1]]
    assert B.moe_balance_scratch_bytes(B.make_shape(T[5], 256, 128, E, 2), S + 1) >= sizes[5]
