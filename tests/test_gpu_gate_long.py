"""The gate over batches so long that a wave takes two batches of tokens: masked rows, rows that
are not finite, rows of equal and of nearly equal scores in both batches of a wave and in the
last, partly filled ones. Every row equals, bit for bit, what the same rows give in short calls (one batch
a wave, the same arithmetic), and rows from the whole range equal the oracle's: ids
exactly, weights and gradients within the bounds of test_gpu_gate.py."""
import numpy as np
import pytest
import torch

from grouped_gemm_02_amd import inputs
from oracle import moe_gate as og

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-5
SHORT = 10_007   # tokens of a short call

# T, E, k, score, bias, renorm, groups, kept, top, mask
LONG = [
    (65543, 256, 8, "sigmoid", True, True, 8, 4, 2, True),
    (65543, 256, 8, "softmax", True, False, 8, 4, 1, True),
    (65539, 256, 12, "sigmoid", True, True, 1, 1, 1, False),
    (65537, 256, 16, "softmax", False, False, 1, 1, 1, True),
    (70001, 128, 8, "softmax", True, True, 1, 1, 1, True),
    (65543, 128, 8, "sigmoid", True, True, 4, 2, 2, False),
    (65543, 128, 16, "sigmoid", False, False, 1, 1, 1, True),
    (70001, 64, 4, "sigmoid", True, True, 8, 4, 2, True),
    (65601, 60, 4, "softmax", False, False, 1, 1, 1, True),
    (131071, 30, 3, "sigmoid", True, False, 1, 1, 1, False),
    (70003, 12, 2, "softmax", True, True, 1, 1, 1, True),
    (32771, 512, 8, "sigmoid", True, True, 16, 4, 2, True),
    (32769, 500, 12, "softmax", False, True, 1, 1, 1, True),
    (16389, 1000, 8, "sigmoid", True, True, 1, 1, 1, True),
    (16385, 1024, 14, "softmax", True, False, 1, 1, 1, False),
    # short, with a bias: several tokens a wave, one batch
    (3001, 256, 8, "sigmoid", True, True, 8, 4, 2, True),
]


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _logits(T, E):
    """Spread rows; the others come at strides that share no factor with the tokens of a wave."""
    z = inputs.make_router_logits(T, E, T + E, DEV, 0.5)
    t = torch.arange(T, device=DEV)
    z[t % 19 == 2] = 0.25                                            # equal
    near = t % 7 == 1                                                # values of a few units of a coarse grid
    z[near] = torch.round(z[near] * 4) / 4
    unit = t % 23 == 4                                               # neighbours in fp32
    z[unit] = torch.nextafter(z[unit][:, :1].expand(-1, E).contiguous(), z[unit])
    z[t % 29 == 6, E // 3] = torch.nan
    z[t % 31 == 8, E - 1] = torch.inf
    z[t % 37 == 9] = -torch.inf
    z[t % 11 == 3, : E // 2] = -torch.inf
    z[-3:] = z[-6:-3].clone()
    return z


@pytest.mark.parametrize("T,E,k,score,bias,renorm,G,L,top,masked", LONG)
def test_long_batches(B, T, E, k, score, bias, renorm, G, L, top, masked):
    print(f"case long T={T} E={E} k={k} {score} bias={bias} renorm={renorm} G={G} L={L} top={top} mask={masked}", flush=True)
    z = _logits(T, E)
    g = torch.Generator().manual_seed(E)
    b = (0.2 if score == "sigmoid" else 0.5 / E) * torch.randn((E,), generator=g).to(DEV) if bias else None
    mask = (torch.rand((T,), generator=g) > 0.2).to(torch.uint8).to(DEV) if masked else None
    p = B.make_gate_params(score, renorm=renorm, groups=G, groups_kept=L, group_top=top, scale=1.5)
    shape = lambda n: B.make_shape(n, 256, 128, E, k)  # noqa: E731
    idx = torch.full((T + 5, k), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T + 5, k), 7.5, device=DEV)
    B.gate(shape(T), p, z, b, mask, idx, w)
    assert (idx[T:] == 77).all() and (w[T:] == 7.5).all()
    idx, w = idx[:T], w[:T]
    dw = torch.randn((T, k), generator=g).to(DEV)
    d = torch.full((T + 1, E), 7.5, device=DEV)
    B.gate_bwd(shape(T), p, z, idx, dw, d)
    assert (d[T] == 7.5).all()
    bits = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
    for at in range(0, T, SHORT):
        n = min(SHORT, T - at)
        i, v = B.gate(shape(n), p, z[at:at + n], b, None if mask is None else mask[at:at + n].clone())
        assert torch.equal(i, idx[at:at + n]) and torch.equal(bits(v), bits(w[at:at + n])), at
        s = B.gate_bwd(shape(n), p, z[at:at + n], i, dw[at:at + n])
        assert torch.equal(bits(s), bits(d[at:at + n])), at
    pick = np.random.default_rng(T).choice(T, 700, replace=False)
    rows = torch.tensor(np.unique(np.concatenate([np.arange(40), pick, np.arange(T - 40, T)])), device=DEV)
    n = lambda t: None if t is None else t[rows].cpu().numpy()  # noqa: E731
    zr, ir, wr = n(z), n(idx), n(w).astype(np.float64)
    ri, rw = og.choose(zr, k, score, renorm, None if b is None else b.cpu().numpy(), G, L, top, 1.5, n(mask))
    assert np.array_equal(ir, ri)
    assert np.array_equal(np.isnan(wr), np.isnan(rw))
    f = ~np.isnan(rw)
    most = np.max(np.abs(np.where(f, rw, 0)), axis=1, keepdims=True)
    assert np.all(np.abs(np.where(f, wr - rw, 0)) <= TOL * most + 1e-38)
    ok = ~np.isnan(zr).any(1) & ~np.isposinf(zr).any(1)
    want = og.choose_backward(zr[ok], ri[ok], n(dw)[ok], score, renorm, 1.5)
    size = 1.5 * np.max(np.abs(n(dw)[ok]), axis=1, keepdims=True)
    assert np.all(np.abs(n(d)[ok].astype(np.float64) - want) <= TOL * size + 1e-38)
