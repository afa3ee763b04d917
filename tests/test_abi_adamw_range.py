"""The range of AdamW's eps: checked before anything reaches the GPU."""
import ctypes
import math
import os

import pytest

from tests.helpers import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")


@pytest.mark.parametrize("eps,status", [(0.0, 0), (2.0 ** -126, 0), (1e-8, 0), (1.0, 0), (2.0 ** 100, 0),
                                        (1e-38, 2), (1e-40, 2), (1e-60, 2), (5e-324, 2), (2.0 ** 101, 2), (3e38, 2), (1e300, 2),
                                        (-1e-8, 2), (-1e-60, 2), (math.nan, 2), (math.inf, 2)])
def test_eps_is_zero_or_a_number_whose_reciprocal_is_one(eps, status):
    from grouped_gemm_02_amd import binding as B
    p = B.moe_adamw_params(1e-3, 0.9, 0.999, eps, 0.1, 0, 0, 0, 1, 0)
    assert B.lib().moe_adamw_step(ctypes.byref(p), None, 0, None, None, None) == status   # no tensors: the checks alone
