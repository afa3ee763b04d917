"""Ends of the documented ranges of the optimizer's entry points, on the host:
what is inside reaches the check of the scratch (status 6), what is outside
does not."""
import ctypes

import pytest

from tests.test_abi_train_cpu import B, P, _call, pytestmark  # noqa: F401


@pytest.mark.parametrize("R,C", [(1, 1), (3, 1), (7, 9), (1000, 777), (16384, 16383), (16384, 16384)])
def test_stacks_up_to_the_element_limit(B, R, C):
    """E R C < 2^40, whether or not R C divides it."""
    most = ((1 << 40) - 1) // (R * C)
    assert _call(B, "moe_orthogonalize", B.make_ortho_shape(most, R, C), P, P, P, 0, None) == 6
    assert _call(B, "moe_orthogonalize", B.make_ortho_shape(most + 1, R, C), P, P, P, 0, None) == 2
    assert B.moe_ortho_workspace_size(B.make_ortho_shape(most, R, C)) > 0
