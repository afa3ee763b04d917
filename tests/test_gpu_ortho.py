"""GPU parity of moe_orthogonalize and moe_muon_step against the float64
oracle, matrix by matrix in the Frobenius norm. The bound, from the formats:
the bf16 result is off by at most 2^-8 of each element (3.9e-3); each of five
steps rounds the products' operands to fp16, 2^-11 at most and 2^-11 / sqrt(3)
in the mean square, times |B| <= 2.8, independently: sqrt(5) * 2.8 * 2^-11 /
sqrt(3) = 1.8e-3. Together below TOL = 6e-3."""
import numpy as np
import pytest
import torch

from oracle import moe_ortho as oo

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 6e-3


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _grad(E, R, C, dtype, seed, rank=None):
    g = torch.Generator().manual_seed(seed)
    r = rank or max(R, C)
    G = torch.randn((E, R, r), generator=g) @ torch.randn((E, r, C), generator=g)
    G = G * 10.0 ** torch.randn((E, 1, 1), generator=g)
    return G.to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(DEV)


def _f64(t):
    return t.double().cpu().numpy()


def _off(got, want):
    """Largest Frobenius error of a matrix, relative to it."""
    out = 0.0
    for a, b in zip(got, want):
        n = np.linalg.norm(b)
        d = np.linalg.norm(a - b)
        out = max(out, d / n if n else (0.0 if d == 0 else np.inf))
    return out


CASES = [
    # (E, R, C, dtype, rank, steps, coeffs)
    (3, 1, 1, "bf16", None, 5, oo.COEFFS),
    (2, 1, 300, "bf16", None, 5, oo.COEFFS),
    (2, 300, 1, "f32", None, 5, oo.COEFFS),
    (3, 5, 7, "f32", None, 5, oo.COEFFS),
    (4, 16, 200, "bf16", 3, 5, oo.COEFFS),
    (2, 64, 64, "bf16", None, 5, oo.COEFFS),
    (3, 127, 129, "bf16", None, 5, oo.COEFFS),
    (2, 128, 256, "bf16", 1, 5, oo.COEFFS),
    (2, 256, 128, "bf16", 10, 5, oo.COEFFS),
    (2, 130, 257, "f32", 40, 5, oo.COEFFS),
    (2, 256, 256, "bf16", None, 5, oo.COEFFS),
    (1, 500, 333, "bf16", None, 5, oo.COEFFS),
    (1, 333, 1000, "f32", 100, 5, oo.COEFFS),
    (2, 640, 512, "bf16", None, 5, oo.COEFFS),
    (2, 200, 384, "bf16", None, 1, oo.COEFFS),
    (2, 384, 200, "bf16", None, 2, oo.COEFFS),
    (2, 200, 384, "f32", None, 6, oo.COEFFS),
    (2, 150, 150, "bf16", None, 8, (1.5, -0.5, 0.0)),
    (2, 256, 256, "bf16", 1, 5, oo.COEFFS),
    (2, 256, 768, "bf16", 1, 5, oo.COEFFS),
    (1, 777, 400, "f32", 1, 5, oo.COEFFS),
    (1, 200, 299, "bf16", None, 2, oo.COEFFS),
    (1, 16384, 130, "bf16", None, 5, oo.COEFFS),
    (2, 334, 3542, "bf16", None, 5, oo.COEFFS),       # X X^T in parts, the last one shorter
    (1, 1030, 140, "f32", None, 5, oo.COEFFS),        # two parts
    (3, 400, 1300, "bf16", 1, 5, oo.COEFFS),
    (1, 40, 16384, "f32", None, 5, oo.COEFFS),
    (2, 200, 384, "bf16", None, 3, (1.5, -0.5, 0.0)),
    (1, 200, 300, "bf16", None, 2, oo.COEFFS),
    (1, 200, 300, "f32", 20, 3, (2.0, -1.5, 0.5)),
]


@pytest.mark.parametrize("E,R,C,dtype,rank,steps,coeffs", CASES)
def test_orthogonalize_matches_oracle(B, E, R, C, dtype, rank, steps, coeffs):
    print(f"case ortho E={E} R={R} C={C} {dtype} rank={rank} steps={steps}", flush=True)
    G = _grad(E, R, C, dtype, E + R + C, rank)
    s = B.make_ortho_shape(E, R, C, steps=steps, grad=dtype, coeffs=coeffs)
    buf = B.OrthoBuffers.allocate(s)
    buf.ws.fill_(0xFF)
    U = torch.full((E, R, C), 9.0, dtype=torch.bfloat16, device=DEV)
    B.orthogonalize(buf, G, U)
    torch.cuda.synchronize()
    err = _off(_f64(U), oo.orthogonalize(_f64(G), steps, coeffs))
    print(f"  off {err:.2e}", flush=True)
    assert err <= TOL


def test_zero_nan_and_extreme_matrices(B):
    """Zeros give zeros; NaN and infinity stay in their matrix; magnitudes
    whose squares leave fp32 are fine; eps as given."""
    E, R, C = 8, 96, 160
    G = _grad(E, R, C, "bf16", 2)
    G[1] = 0
    G[2, 5, 7] = float("nan")
    G[3, 95, 159] = float("inf")
    G[4] = G[0] * 1e30
    G[5] = G[0] * 1e-30
    G[6] = 0
    G[6, 3, 4] = 2.0
    s = B.make_ortho_shape(E, R, C, eps=0.0)
    U = B.orthogonalize(B.OrthoBuffers.allocate(s), G)
    got, want = _f64(U), oo.orthogonalize(_f64(G), eps=0.0)
    assert not got[1].any() and np.isnan(got[2]).all() and np.isnan(got[3]).all()
    rest = [0, 4, 5, 6, 7]
    assert _off(got[rest], want[rest]) <= TOL
    s = B.make_ortho_shape(1, R, C, eps=3.0 * float(G[0].float().norm()))
    assert _off(_f64(B.orthogonalize(B.OrthoBuffers.allocate(s), G[:1])), oo.orthogonalize(_f64(G[:1]), eps=s.eps)) <= TOL


@pytest.mark.parametrize("R,C", [(40, 70), (150, 290)])   # either path
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_magnitudes_at_the_ends_of_the_types(B, R, C, dtype):
    """Largest elements near the type's largest, near its smallest normal and
    among its subnormals (eps 0); a norm far below eps."""
    print(f"case ortho magnitudes R={R} C={C} {dtype}", flush=True)
    G = _grad(4, R, C, "f32", 4)
    G = G / G.abs().amax(dim=(1, 2), keepdim=True)
    G = (G.double() * torch.tensor([3.3e38, 2e-38, 2e-39, 1e-10], device=DEV, dtype=torch.float64).view(4, 1, 1))
    G = G.float().to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    for eps, rows in ((0.0, slice(0, 3)), (1e-7, slice(3, 4))):
        s = B.make_ortho_shape(G[rows].shape[0], R, C, grad=dtype, eps=eps)
        U = B.orthogonalize(B.OrthoBuffers.allocate(s), G[rows].clone())
        assert _off(_f64(U), oo.orthogonalize(_f64(G[rows]), eps=s.eps)) <= TOL


@pytest.mark.parametrize("coeffs,steps", [((17.0, 0.0, 0.0), 2), ((2.0, -0.3, 0.0), 4), ((2.5, -2.0, 0.5), 5)])
def test_polynomials_that_let_small_matrices_grow(B, coeffs, steps):
    """Singular values well past 1, elements below 2."""
    print(f"case ortho polynomial {coeffs} {steps}", flush=True)
    G = torch.zeros((2, 96, 128), device=DEV)
    G[0, 5] = 1.0
    G[1] = torch.randn((96, 128), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    G = G.bfloat16()
    s = B.make_ortho_shape(2, 96, 128, steps=steps, coeffs=coeffs)
    U = B.orthogonalize(B.OrthoBuffers.allocate(s), G)
    want = oo.orthogonalize(_f64(G), steps, tuple(float(np.float32(c)) for c in coeffs))
    assert np.isfinite(want).all() and _off(_f64(U), want) <= TOL


def test_matrices_do_not_depend_on_their_stack(B):
    """A matrix gives the same bits alone, in a stack, in place, and again."""
    for E, R, C in ((6, 200, 300), (5, 64, 100), (5, 300, 200)):
        G = _grad(E, R, C, "bf16", 3)
        buf = B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C))
        U = B.orthogonalize(buf, G).clone()
        assert torch.equal(U, B.orthogonalize(buf, G))
        one = B.OrthoBuffers.allocate(B.make_ortho_shape(1, R, C))
        for e in range(E):
            assert torch.equal(B.orthogonalize(one, G[e:e + 1].contiguous())[0], U[e])
        H = G.clone()
        B.orthogonalize(buf, H, H)
        assert torch.equal(H, U)


def test_past_32_bits(B):
    """More than 2^31 elements, in more than one group: the last matrices are
    the bits they are alone."""
    R, C = 1200, 900
    E = (1 << 31) // (R * C) + 3
    G = _grad(3, R, C, "bf16", 5)
    big = torch.empty((E, R, C), dtype=torch.bfloat16, device=DEV)
    big[:] = G[0]
    big[E - 2:] = G[1:]
    U = B.orthogonalize(B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C)), big)
    few = B.orthogonalize(B.OrthoBuffers.allocate(B.make_ortho_shape(3, R, C)), G)
    assert torch.equal(U[E - 2:], few[1:])
    assert torch.equal(U[0], few[0]) and torch.equal(U[E - 3], few[0]) and torch.equal(U[E // 2], few[0])


BIG = [
    # (E, R, C, dtype): enough matrices for the large tiles, sides that end inside one
    (200, 300, 500, "bf16"),
    (200, 500, 300, "f32"),
    (180, 130, 700, "bf16"),
    (520, 128, 256, "bf16"),
    (1100, 24, 33, "f32"),     # more than a group of small matrices
    (130, 640, 385, "bf16"),
]


@pytest.mark.parametrize("E,R,C,dtype", BIG)
def test_large_stacks_match_oracle(B, E, R, C, dtype):
    """A stack that runs in large tiles: matrices from its ends and its middle."""
    print(f"case ortho stack E={E} R={R} C={C} {dtype}", flush=True)
    few = _grad(4, R, C, dtype, 11, rank=min(R, C) // 2)
    G = few[torch.arange(E, device=DEV) % 3].contiguous()
    G[E // 2 + 1] = few[3]
    G[E - 1] = few[3]
    U = B.orthogonalize(B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C, grad=dtype)), G)
    want = oo.orthogonalize(_f64(few))
    assert _off(_f64(U[:3]), want[:3]) <= TOL
    assert _off(_f64(U[E - 1:]), want[3:]) <= TOL
    same = torch.arange(E, device=DEV) % 3
    same[E // 2 + 1] = same[E - 1] = 3
    ref = torch.cat([U[:3], U[E - 1:]])
    assert torch.equal(U, ref[same])


@pytest.mark.parametrize("master", [False, True])
def test_large_stack_of_weights(B, master):
    E, R, C = 200, 500, 301
    few = _grad(2, R, C, "bf16", 5, rank=200)
    G = few[torch.arange(E, device=DEV) % 2].contiguous()
    g = torch.Generator().manual_seed(1)
    mast = (0.05 * torch.randn((1, R, C), generator=g)).to(DEV).expand(E, R, C).contiguous()
    W = mast.to(torch.bfloat16)
    mom = torch.zeros_like(mast)
    want_m, want = oo.muon_step(_f64(few), np.zeros((2, R, C)), _f64(mast[:2] if master else W[:2]), 0.02, 0.9, 0.1, 2.0,
                                True)
    before = _f64(mast[:2] if master else W[:2]) * (1 - 0.02 * 0.1)
    B.muon_step(B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C)), G, mom, W, lr=0.02, momentum_coef=0.9,
                weight_decay=0.1, scale=2.0, nesterov=True, master=mast if master else None)
    for k in (0, E - 2):
        got = _f64((mast if master else W)[k:k + 2])
        tol = (2.0 ** -22 if master else 2.0 ** -8) * np.linalg.norm(want) + TOL * np.linalg.norm(want - before)
        assert np.linalg.norm(got - want) <= tol
        assert _off(_f64(mom[k:k + 2]), want_m) <= 2.0 ** -22


MUON = [
    # (E, R, C, dtype, nesterov, master)
    (2, 100, 60, "bf16", True, False),
    (2, 60, 100, "bf16", False, True),
    (2, 256, 128, "f32", True, True),
    (1, 300, 513, "f32", False, False),
    (3, 7, 5, "bf16", True, True),
]


@pytest.mark.parametrize("E,R,C,dtype,nesterov,master", MUON)
def test_muon_steps_match_oracle(B, E, R, C, dtype, nesterov, master):
    """Three steps in a row. Momentum: one fused multiply-add a step, 2^-23.
    Weights: each step's bf16 rounding 2^-8, master weights 2^-23, and what
    the orthogonalisation is off by, times lr * scale."""
    print(f"case muon E={E} R={R} C={C} {dtype} nesterov={nesterov} master={master}", flush=True)
    lr, mu, wd, scale = 0.02, 0.95, 0.1, 2.0
    g = torch.Generator().manual_seed(R)
    mast = (0.05 * torch.randn((E, R, C), generator=g)).to(DEV)
    W = mast.to(torch.bfloat16)
    mom = (0.1 * torch.randn((E, R, C), generator=g)).to(DEV)
    buf = B.OrthoBuffers.allocate(B.make_ortho_shape(E, R, C, grad=dtype))
    m64 = _f64(mom)
    for k in range(3):
        G = _grad(E, R, C, dtype, k, rank=30)
        before = _f64(mast if master else W)
        m64, want = oo.muon_step(_f64(G), _f64(mom), before, lr, mu, wd, scale, nesterov)
        B.muon_step(buf, G, mom, W, lr=lr, momentum_coef=mu, weight_decay=wd, scale=scale, nesterov=nesterov,
                    master=mast if master else None)
        torch.cuda.synchronize()
        assert _off(_f64(mom), m64) <= 2.0 ** -22
        upd = np.linalg.norm(want - before * (1 - lr * wd))
        if master:
            assert np.linalg.norm(_f64(mast) - want) <= 2.0 ** -22 * np.linalg.norm(want) + TOL * upd
            assert torch.equal(W, mast.to(torch.bfloat16))
        else:
            assert np.linalg.norm(_f64(W) - want) <= 2.0 ** -8 * np.linalg.norm(want) + TOL * upd
