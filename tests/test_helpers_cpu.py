"""The error measures of the test suite reject what is not a number."""
import math

import numpy as np
import pytest

from tests.helpers import max_matrix_err, max_rel_err


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_matrix_error_rejects_non_finite(bad):
    ref = np.ones((3, 4, 5))
    for e in range(3):
        got = ref.copy()
        got[e, 1, 2] = bad
        assert max_matrix_err(got, ref) == math.inf
    assert max_matrix_err(np.full_like(ref, bad), ref) == math.inf
    assert max_matrix_err(np.full_like(ref, bad), 0 * ref) == math.inf
    assert not max_rel_err(np.full_like(ref, bad), ref) <= 1.0


def test_matrix_error_is_that_of_the_worst_matrix():
    ref = np.ones((3, 2, 2))
    got = ref.copy()
    got[1] *= 1.5
    got[2] *= 1.25
    assert max_matrix_err(got, ref) == pytest.approx(0.5)
    assert max_matrix_err(ref, ref) == 0.0
    assert max_matrix_err(0 * ref, 0 * ref) == 0.0
    assert max_matrix_err(ref, 0 * ref) == math.inf
