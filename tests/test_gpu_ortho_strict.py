"""The cases of test_gpu_ortho.py measured by helpers.max_matrix_err, which a
NaN or an infinity cannot pass (Python's max(0.0, nan) is 0.0), and steps on
the weights over more than one group of matrices. Bounds as derived there."""
import numpy as np
import pytest
import torch

from oracle import moe_ortho as oo
from tests import test_gpu_ortho as base
from tests.helpers import max_matrix_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = base.TOL
B = base.B


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(base, "_off", max_matrix_err)


@pytest.mark.parametrize("E,R,C,dtype,rank,steps,coeffs", base.CASES)
def test_orthogonalize(B, E, R, C, dtype, rank, steps, coeffs):
    base.test_orthogonalize_matches_oracle(B, E, R, C, dtype, rank, steps, coeffs)


def test_beside_zero_nan_and_extreme_matrices(B):
    base.test_zero_nan_and_extreme_matrices(B)


@pytest.mark.parametrize("R,C", [(40, 70), (150, 290)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_magnitudes(B, R, C, dtype):
    base.test_magnitudes_at_the_ends_of_the_types(B, R, C, dtype)


@pytest.mark.parametrize("coeffs,steps", [((17.0, 0.0, 0.0), 2), ((2.0, -0.3, 0.0), 4), ((2.5, -2.0, 0.5), 5)])
def test_polynomials_that_grow(B, coeffs, steps):
    base.test_polynomials_that_let_small_matrices_grow(B, coeffs, steps)


@pytest.mark.parametrize("E,R,C,dtype", base.BIG)
def test_large_stacks(B, E, R, C, dtype):
    base.test_large_stacks_match_oracle(B, E, R, C, dtype)


@pytest.mark.parametrize("master", [False, True])
def test_large_stack_of_weights(B, master):
    base.test_large_stack_of_weights(B, master)


@pytest.mark.parametrize("E,R,C,dtype,nesterov,master", base.MUON)
def test_muon_steps(B, E, R, C, dtype, nesterov, master):
    base.test_muon_steps_match_oracle(B, E, R, C, dtype, nesterov, master)


GROUPS = [
    # (E, R, C): a group is 4096 matrices of this size, 1024 of smaller side up to 128
    (4099, 130, 140),
    (4099, 140, 130),
    (1027, 20, 33),
    (1027, 33, 20),
]


@pytest.mark.parametrize("E,R,C", GROUPS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("master", [False, True])
def test_steps_on_weights_of_more_than_one_group(B, E, R, C, dtype, master):
    """Matrices of both groups, each with a gradient, a momentum and weights
    of its own."""
    print(f"case muon groups E={E} R={R} C={C} {dtype} master={master}", flush=True)
    lr, mu, wd, scale = 0.02, 0.9, 0.1, 2.0
    g = torch.Generator(device=DEV).manual_seed(E + R)
    n = lambda: torch.randn((E, R, C), generator=g, device=DEV)  # noqa: E731
    G = n().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    mom, mast = 0.5 * n(), 0.05 * n()
    W = mast.bfloat16()
    some = [0, 1, E // 2, E - 5, E - 4, E - 3, E - 2, E - 1]   # the last group is the last three
    g64, m64, old = (t[some].double().cpu().numpy() for t in (G, mom, mast if master else W))
    want_m, want = oo.muon_step(g64, m64, old, lr, mu, wd, scale, True)
    B.muon_step(B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C, grad=dtype)), G, mom, W, lr=lr, momentum_coef=mu,
                weight_decay=wd, scale=scale, nesterov=True, master=mast if master else None)
    torch.cuda.synchronize()
    got_m, got = (t[some].double().cpu().numpy() for t in (mom, mast if master else W))
    assert max_matrix_err(got_m, want_m) <= 2.0 ** -22
    for k in range(len(some)):
        upd = np.linalg.norm(want[k] - old[k] * (1 - lr * wd))
        size = np.linalg.norm(want[k])
        assert np.linalg.norm(got[k] - want[k]) <= (2.0 ** -22 if master else 2.0 ** -8) * size + TOL * upd, some[k]
    if master:
        assert torch.equal(W, mast.bfloat16())
