"""Gradients of the dense products' activations where P is finite but far from the usual.

With W the unit matrix dX is dP rounded to bf16 (2^-8), and with one row dbias is dP itself.
The sigmoid s is off by 2^-16 of itself where its argument is at most 20 in magnitude (the
argument's few roundings of 2^-24 become 20 * 2^-22, two more units for the power and the
reciprocal). The slopes' terms carry that: s, and |g| s (1 - s) times the argument's own slope.
1 - s is a difference of numbers near 1, off by 2^-23, and 0 from arguments of 17 on: times
what multiplies it, at most 17 (silu) or 45 (GELU at 5.5), 2^-17 for g > 0 covers it. Far from
0 the sigmoid is 0 or 1 exactly, and the slope with it."""
import numpy as np
import pytest
import torch

from oracle import moe_linear as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
# both signs of each: an ordinary range, and beyond the square and the cube of fp32's range
FAR = [1e3, 1e10, 6e12, 1e13, 1.5e19, 2e19, 6e19, 1e25, 1e38, 3.3e38]
NEAR = [0.0, 0.125, 0.5, 1.0, 2.0, 4.0, 5.0]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _n(t):
    return t.double().cpu().numpy()


def _dp(B, act, dY, P):
    """dP of every element: rounded by way of dX, and as it is by way of dbias, a row at a time."""
    M, N = dY.shape
    R = P.shape[1]
    W = torch.eye(R, dtype=torch.bfloat16, device=DEV)
    X = torch.ones((M, R), dtype=torch.bfloat16, device=DEV)
    out = "f32" if dY.dtype == torch.float32 else "bf16"
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, R, act=act, out=out))
    dX, _, db = B.linear_bwd(buf, dY, X, W, P, bias=True)
    rows = [B.linear_bwd(buf, dY[i:i + 1].clone(), None, W, P[i:i + 1].clone(), bias=True, need_dX=False,
                         need_dW=False)[2] for i in range(M)]
    return dX, torch.stack(rows), db


def _slope_error(g, act):
    s = ol._sigmoid(g if act != "gelu" else 2 * ol.A * (g + ol.B * g ** 3))
    inner = np.abs(g) * s * (1 - s) * (1.0 if act != "gelu" else 2 * ol.A * (1 + 3 * ol.B * g * g))
    return 2.0 ** -16 * (s + inner) + 2.0 ** -17 * (g > 0)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_slopes_of_finite_p(B, act, out):
    print(f"case far P {act} {out}", flush=True)
    v = np.array(FAR + NEAR)
    g = torch.tensor(np.concatenate([v, -v])).bfloat16()
    d = torch.tensor([1.0, -3.0, 1e-3, 100.0, 0.0]).to(torch.bfloat16 if out == "bf16" else torch.float32)
    P = g[None, :].expand(len(d), -1).contiguous().to(DEV)
    dY = d[:, None].expand(-1, len(g)).contiguous().to(DEV)
    dX, rows, db = _dp(B, act, dY, P)
    want = ol.slope_times(_n(dY), _n(P), act)
    assert np.isfinite(want).all()
    e = np.abs(_n(dY)) * (0.0 if act == "relu" else _slope_error(_n(P), act))
    assert np.all(np.abs(_n(rows) - want) <= e + 2.0 ** -24 * np.abs(want))
    assert np.all(np.abs(_n(dX) - want) <= e + 2.0 ** -8 * (np.abs(want) + e))
    assert np.all(np.abs(_n(db) - want.sum(0)) <= e.sum(0) + 8 * 2.0 ** -24 * np.abs(want).sum(0))


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_pairs_of_finite_p(B, out):
    """Gate and up parts whose products with dY leave fp32's range before a factor of 0 meets
    them, or where the gradient itself does not."""
    print(f"case far pairs {out}", flush=True)
    v = FAR + [1.0, 4.0]
    g = np.array(v + [-x for x in v] + [0.0])
    u = np.array([1.0, -1e19, 1e25, -1e38, 3.3e38, 0.0])
    G, U = (torch.tensor(t.ravel()).bfloat16() for t in np.meshgrid(g, u))
    d = torch.tensor([1.0, -100.0, 1e-3, 1e5, 0.25]).to(torch.bfloat16 if out == "bf16" else torch.float32)
    P = torch.cat([G, U])[None, :].expand(len(d), -1).contiguous().to(DEV)
    dY = d[:, None].expand(-1, len(G)).contiguous().to(DEV)
    dX, rows, _ = _dp(B, "swiglu", dY, P)
    x, (gg, uu) = np.abs(_n(dY)), np.split(_n(P), 2, axis=1)
    want = ol.slope_times(_n(dY), _n(P), "swiglu")
    e = np.concatenate([x * np.abs(uu) * _slope_error(gg, "silu"), 2.0 ** -16 * x * np.abs(gg) * ol._sigmoid(gg)], axis=1)
    # the largest number of bf16 is 2^-8 of itself below fp32's
    big = float(torch.finfo(torch.float32).max)
    inside, beyond = np.abs(want) < big * (1 - 2.0 ** -7), np.abs(want) > big * (1 + 2.0 ** -7)
    off = np.abs(_n(rows) - want)[inside]
    assert np.all(off <= (e + 3 * 2.0 ** -24 * np.abs(want))[inside] + 1e-37)
    assert beyond.any() and np.all(_n(rows)[beyond] == np.sign(want[beyond]) * np.inf)
    # an infinity in dP meets the unit matrix' zeros: rows without one
    whole = inside.all(1)
    assert whole.sum() >= 2
    off = np.abs(_n(dX) - want)[whole]
    assert np.all(off <= (e + 2.0 ** -8 * (np.abs(want) + e) + 3 * 2.0 ** -24 * np.abs(want))[whole] + 1e-37)
