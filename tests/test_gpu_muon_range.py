"""The update of the weights where its elements are very small or large, against
the float64 oracle: on fp32 master weights, which show it without a bf16
rounding. The bound, from the formats: the products' roundings of five steps
as derived in test_gpu_ortho.py, 1.8e-3 of the update's norm, the pairs of bf16
that carry it 2^-17 of each element, the master weights 2^-24."""
import numpy as np
import pytest
import torch

from oracle import moe_ortho as oo
from tests import test_gpu_ortho as base
from tests.helpers import max_matrix_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = base.B
TOL_UPDATE = 1.8e-3 + 2.0 ** -17 + 2.0 ** -23


def _update(B, G, W, master, shape_kw, **kw):
    """The step on weights of zero; (what they became, the oracle's)."""
    E, R, C = G.shape
    dtype = "bf16" if G.dtype == torch.bfloat16 else "f32"
    s = B.make_ortho_shape(E, R, C, grad=dtype, **shape_kw)
    mom = torch.zeros((E, R, C), device=DEV)
    buf = B.OrthoBuffers.allocate(s)
    buf.ws.fill_(0xFF)
    B.muon_step(buf, G, mom, W, momentum_coef=0.0, weight_decay=0.0, nesterov=False, master=master, **kw)
    torch.cuda.synchronize()
    U = oo.orthogonalize(base._f64(G), s.steps, (s.a, s.b, s.c), s.eps)
    return base._f64(W if master is None else master), -float(np.float32(kw["lr"])) * float(np.float32(kw["scale"])) * U


SHAPES = [(1, 512, 8192), (1, 8192, 512), (1, 128, 16384), (1, 16384, 100)]   # either path, wide and tall


@pytest.mark.parametrize("E,R,C", SHAPES)
def test_gradients_far_below_eps(B, E, R, C):
    """|G| = eps / 9e4: the update's elements are a few 1e-6."""
    print(f"case muon below eps {E} {R} {C}", flush=True)
    G = torch.randn((E, R, C), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    G = (G / G.norm() * (1e-7 / 9e4)).contiguous()
    master, W = torch.zeros_like(G), torch.zeros_like(G).bfloat16()
    got, want = _update(B, G, W, master, {}, lr=1.0, scale=2.0 ** 16)
    err = max_matrix_err(got, want)
    print(f"  off {err:.2e}", flush=True)
    assert err <= TOL_UPDATE
    assert torch.equal(W, master.bfloat16())


@pytest.mark.parametrize("E,R,C", [(2, 150, 140), (2, 140, 300)])
@pytest.mark.parametrize("with_master", [False, True])
def test_steep_polynomials(B, E, R, C, with_master):
    """Elements of the update past 65504."""
    print(f"case muon steep {E} {R} {C}", flush=True)
    G = base._grad(E, R, C, "bf16", 3)
    W = torch.zeros((E, R, C), dtype=torch.bfloat16, device=DEV)
    master = torch.zeros((E, R, C), device=DEV) if with_master else None
    got, want = _update(B, G, W, master, dict(steps=1, coeffs=(1e8, 0.0, 0.0)), lr=0.5, scale=1e-7)
    assert max_matrix_err(got, want) <= TOL_UPDATE + (0 if with_master else 2.0 ** -8)


@pytest.mark.parametrize("E,R,C,dtype", [(2, 64, 100, "bf16"), (2, 100, 64, "f32"), (3, 127, 33, "f32"),
                                         (2, 256, 300, "bf16"), (2, 300, 256, "f32"), (200, 300, 500, "bf16"),
                                         (200, 500, 300, "f32"), (1, 1000, 777, "f32")])
def test_updates_of_master_weights(B, E, R, C, dtype):
    print(f"case muon master {E} {R} {C} {dtype}", flush=True)
    few = base._grad(min(E, 3), R, C, dtype, 5)
    G = few[torch.arange(E, device=DEV) % few.shape[0]].contiguous()
    master = torch.zeros((E, R, C), device=DEV)
    W = torch.zeros((E, R, C), dtype=torch.bfloat16, device=DEV)
    s = B.make_ortho_shape(E, R, C, grad=dtype)
    B.muon_step(B.OrthoBuffers.allocate(s), G, torch.zeros_like(master), W, lr=1.0, scale=1.0, momentum_coef=0.0,
                nesterov=False, master=master)
    torch.cuda.synchronize()
    err = max_matrix_err(-base._f64(master[:few.shape[0]]), oo.orthogonalize(base._f64(few)))
    print(f"  off {err:.2e}", flush=True)
    assert err <= TOL_UPDATE
    assert torch.equal(master[E - 1], master[(E - 1) % few.shape[0]]) and torch.equal(W, master.bfloat16())


RANK_ONE = [(2, 200, 384, "f32"), (2, 384, 200, "bf16"), (2, 100, 384, "f32"), (2, 384, 100, "bf16")]


@pytest.mark.parametrize("E,R,C,dtype", RANK_ONE)
def test_updates_of_rank_one(B, E, R, C, dtype):
    """The fp32 sum of gradient and momentum enters as fp16 and an E4M3 remainder
    of it: in the mean square off by at most 2^-11 / sqrt(3) times 2^-4 / sqrt(3)
    of an element (tiled path), which the directions that a matrix of rank one
    lacks grow 485-fold: 4.9e-3, with the products' 1.8e-3 below TOL."""
    print(f"case muon rank one {E} {R} {C} {dtype}", flush=True)
    G = base._grad(E, R, C, dtype, 9, rank=1)
    master, W = torch.zeros((E, R, C), device=DEV), torch.zeros((E, R, C), dtype=torch.bfloat16, device=DEV)
    got, want = _update(B, G, W, master, {}, lr=1.0, scale=1.0)
    err = max_matrix_err(got, want)
    print(f"  off {err:.2e}", flush=True)
    assert err <= base.TOL
