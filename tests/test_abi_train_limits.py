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


@pytest.mark.parametrize("kw,status", [(dict(), 6), (dict(lr=1e30, scale=1e30), 2), (dict(lr=-1e30, scale=1e30), 2),
                                       (dict(lr=1e30, weight_decay=1e30), 2), (dict(lr=1e19, scale=1e19), 6),
                                       (dict(lr=1e19, weight_decay=-1e19), 6), (dict(lr=0.0, scale=3e38), 6)])
def test_products_of_parameters_are_finite(B, kw, status):
    """lr scale and lr weight_decay past fp32 would make weights NaN where the
    update is zero."""
    a = dict(lr=0.1, mu=0.9, weight_decay=0.0, scale=1.0, nesterov=1, reserved=0)
    a.update(kw)
    p = B.moe_muon_params(**a)
    assert _call(B, "moe_muon_step", B.make_ortho_shape(2, 100, 64), ctypes.byref(p), P, P, P, P, P, 0, None) == status
