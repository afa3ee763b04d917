"""GPU parity of moe_gate and moe_gate_bwd against the float64 oracle.

Ids are compared exactly: both sides choose by 64-bit values, and the inputs'
neighbours differ by far more than 2^-50 or are equal. Weights: the value is
computed in fp32 or better from a score whose exponential, sum and division are each off
by a few units of 2^-24 (at most 16 of them together): 2^-20 of the value, and an
exponent's argument of magnitude a adds a 2^-24 of itself, a <= 104 before the score
is below fp32's range: TOL = 1e-5 relative to the row's largest. Gradients: products
of such values and a difference d - <p, d>, relative to scale * the row's largest |d|."""
import numpy as np
import pytest
import torch

from grouped_gemm_02_amd import inputs
from oracle import moe_gate as og

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-5


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _bias(E, seed, size=0.1):
    return size * torch.randn((E,), generator=torch.Generator().manual_seed(seed)).to(DEV)


def _check(B, z, k, score, renorm, bias=None, G=1, L=None, top=1, scale=1.0, mask=None, seed=0):
    T, E = z.shape
    print(f"case T={T} E={E} k={k} {score} renorm={renorm} bias={bias is not None} G={G} L={L} top={top}", flush=True)
    shape = B.make_shape(T, 256, 128, E, k)
    p = B.make_gate_params(score, renorm=renorm, groups=G, groups_kept=L, group_top=top, scale=scale)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    got = B.gate(shape, p, z, bias, mask, idx, w)
    assert got[0] is idx and got[1] is w
    n = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    ri, rw = og.choose(n(z), k, score, renorm, n(bias), G, L, top, scale, n(mask))
    i, v = n(idx), n(w).astype(np.float64)
    assert np.array_equal(i, ri), np.argwhere(i != ri)[:5]
    assert np.array_equal(np.isnan(v), np.isnan(rw))
    f = ~np.isnan(rw)
    top_w = np.max(np.abs(np.where(f, rw, 0)), axis=1, keepdims=True)
    assert np.all(np.abs(np.where(f, v - rw, 0)) <= TOL * top_w + 1e-38)
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(seed + 9)).to(DEV)
    ok = np.isfinite(n(z)).all(axis=1) | np.isneginf(n(z)).any(axis=1) & ~np.isnan(n(z)).any(axis=1)
    d = B.gate_bwd(shape, p, z, idx, dw, torch.full((T, E), -7.0, device=DEV))
    _compare_bwd(n(d), og.choose_backward(n(z), ri, n(dw), score, renorm, scale), n(dw), scale, ok)
    return idx, w


def _compare_bwd(d, want, dw, scale, rows=None):
    rows = np.ones(len(d), bool) if rows is None else rows
    size = abs(scale) * np.max(np.abs(dw), axis=1, keepdims=True)
    off = np.abs(d.astype(np.float64) - want)[rows]
    assert np.all(off <= TOL * size[rows] + 1e-38), float(np.max(off / size[rows]))


SHAPES = [(2000, 128, 8), (300, 256, 8), (64, 8, 2), (1, 1, 1), (1, 3, 2), (1007, 60, 4), (500, 16, 16), (77, 200, 65),
          (65, 1024, 8), (9, 1024, 1024), (33, 511, 12), (40, 257, 7), (130, 64, 6), (128, 32, 4)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_matches_oracle(B, T, E, k, score):
    z = inputs.make_router_logits(T, E, T + E, DEV, 0.5)
    for renorm in (True, False):
        _check(B, z, k, score, renorm, scale=2.5 if renorm else 1.0)
        _check(B, z, k, score, renorm, _bias(E, T, 0.2 if score == "sigmoid" else 0.5 / E))


GROUPED = [(400, 256, 8, 8, 4, 2), (300, 128, 4, 4, 1, 1), (200, 64, 6, 8, 3, 2), (100, 60, 4, 5, 2, 2), (90, 60, 12, 5, 1, 1),
           (50, 36, 2, 36, 3, 1), (50, 36, 2, 36, 2, 2), (70, 1024, 8, 64, 4, 2), (60, 512, 8, 16, 2, 2), (33, 96, 5, 3, 2, 2),
           (20, 256, 128, 8, 4, 2), (64, 16, 2, 2, 1, 2), (300, 160, 6, 8, 3, 1)]


@pytest.mark.parametrize("T,E,k,G,L,top", GROUPED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_match_oracle(B, T, E, k, G, L, top, score):
    z = inputs.make_router_logits(T, E, T * E, DEV, 0.3)
    mask = (torch.arange(T, device=DEV) % 7 != 3).to(torch.uint8)
    _check(B, z, k, score, True, _bias(E, E, 0.2 if score == "sigmoid" else 0.5 / E), G, L, top, 2.5, mask)
    _check(B, z, k, score, False, None, G, L, top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,L,top", [(128, 1, 1, 1), (256, 8, 4, 2), (60, 5, 2, 2), (256, 8, 2, 1), (1000, 1, 1, 1)])
def test_ties_go_to_the_lower_id(B, score, E, G, L, top):
    """Logits of a few values each, and rows of one value alone, without a bias, with a
    constant one (which changes nothing) and with one that repeats."""
    T, k = 200, 6
    g = torch.Generator().manual_seed(E)
    z = (torch.randint(0, 5, (T, E), generator=g).float() * 0.5).to(DEV)
    z[::9] = 0.25
    _check(B, z, k, score, True, None, G, L, top)
    i0, _ = _check(B, z, k, score, True, torch.zeros(E, device=DEV), G, L, top)
    _check(B, z, k, score, False, (torch.arange(E, device=DEV) % 4).float() * 0.125, G, L, top)
    if G == 1:
        assert torch.equal(i0[0].cpu(), torch.arange(k, dtype=torch.int32))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbours_below_fp32(B, score):
    """Choices that differ in 64 bits and not in 32: logits one unit apart, where the
    scores round to the same fp32 number, and biases that bring far scores together."""
    T, E, k = 64, 256, 8
    g = torch.Generator().manual_seed(5)
    base = (3.0 + torch.randn((T, 1), generator=g)).float()
    step = torch.randint(0, 40, (T, E), generator=g)
    z = torch.from_numpy(base.numpy() + (step.numpy() * np.spacing(base.numpy())).astype(np.float32)).to(DEV)
    _check(B, z, k, score, True)
    _check(B, z, k, score, True, torch.zeros(E, device=DEV), 8, 3, 2)
    _check(B, z, k, score, True, _bias(E, 4, 1e-7))
    z = torch.randn((T, E), generator=g)
    s = torch.softmax(z[0].double(), 0) if score == "softmax" else torch.sigmoid(z[0].double())
    bias = (0.5 - s).float().to(DEV)   # every choice of row 0 within 2^-24 of 0.5
    _check(B, z.to(DEV), k, score, True, bias)
    _check(B, z.to(DEV), k, score, False, bias, 8, 2, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,L,top", [(128, 1, 1, 1), (256, 8, 4, 2), (60, 5, 2, 2), (24, 4, 2, 1)])
def test_rows_with_little_left(B, score, E, G, L, top):
    """Experts off by their logit or their bias, up to all of them; groups with one
    expert left; the type's lowest value; NaN and infinities in their own rows alone."""
    T, k = 96, 4
    z = inputs.make_router_logits(T, E, 3, DEV)
    z[1] = -torch.inf
    z[2, 1:] = -torch.inf
    z[3, :E - 2] = -torch.inf
    z[4] = torch.finfo(torch.float32).min
    z[5, ::2] = torch.finfo(torch.float32).min
    z[6] = 1e30
    z[7] = -1e4 + z[7]
    z[8] = 1e4 + z[8]
    z[9, E // 3] = torch.nan
    z[10, 0] = torch.inf
    z[11, E - 1] = torch.inf
    z[12] = torch.nan
    z[13, : E // 2] = -torch.inf
    z[14, ::3] = -torch.inf
    for renorm in (True, False):
        _check(B, z, k, score, renorm, None, G, L, top)
        b = _bias(E, 8)
        b[0] = -torch.inf
        b[E // 2] = -torch.inf
        _check(B, z, k, score, renorm, b, G, L, top)
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        mask[9:13] = 0   # what is masked is not looked at
        mask[20:40] = 0
        _check(B, z, k, score, renorm, b, G, L, top, 1.0, mask)
    _check(B, z[20:30].contiguous(), k, score, True, torch.full((E,), torch.nan, device=DEV), G, L, top)
    _check(B, z[20:30].contiguous(), k, score, True, torch.full((E,), -torch.inf, device=DEV), G, L, top)


def test_agrees_with_moe_route(B):
    T, E, k = 3000, 128, 8
    z = inputs.make_router_logits(T, E, 17, DEV, 1.2)
    shape = B.make_shape(T, 256, 128, E, k)
    for renorm in (True, False):
        idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
        w = torch.empty((T, k), device=DEV)
        B.moe_route(shape, z, renorm, idx, w)
        i, v = B.gate(shape, B.make_gate_params("softmax", renorm=renorm), z)
        assert torch.equal(i, idx)
        assert torch.allclose(v, w, rtol=TOL, atol=0)
        dw = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).to(DEV)
        a, b = torch.empty_like(z), B.gate_bwd(shape, B.make_gate_params("softmax", renorm=renorm), z, idx, dw)
        B.moe_route_bwd(shape, z, idx, w, dw, renorm, a)
        assert torch.allclose(a, b, rtol=0, atol=TOL * 4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(500, 60, 5), (200, 256, 8), (37, 1000, 20), (3, 1024, 200)])
def test_backward_of_any_ids(B, score, renorm, T, E, k):
    """Ids outside [0, E), an expert named several times, whole rows without one; and
    accumulation into what is there."""
    print(f"case bwd ids T={T} E={E} k={k} {score} {renorm}", flush=True)
    g = torch.Generator().manual_seed(T)
    z = torch.randn((T, E), generator=g)
    idx = torch.randint(-2, E + 2, (T, k), generator=g).to(torch.int32)
    idx[:, 1] = idx[:, 0]
    if k > 3:
        idx[:, 3] = idx[:, 0]
    idx[::5] = -1
    idx[1::5] = E + 5
    idx[2] = torch.iinfo(torch.int32).min
    dw = torch.randn((T, k), generator=g)
    want = og.choose_backward(z.numpy(), idx.numpy(), dw.numpy(), score, renorm, 1.5)
    shape, p = B.make_shape(T, 256, 128, E, k), B.make_gate_params(score, renorm=renorm, scale=1.5)
    d = B.gate_bwd(shape, p, z.to(DEV), idx.to(DEV), dw.to(DEV), torch.full((T, E), torch.nan, device=DEV))
    size = dw.numpy() * np.sqrt(k)   # k slots may fall on one expert
    _compare_bwd(d.cpu().numpy(), want, size, 1.5)
    old = torch.randn((T, E), generator=g)
    acc = old.to(DEV)
    B.gate_bwd(shape, p, z.to(DEV), idx.to(DEV), dw.to(DEV), acc, accumulate=True)
    got = acc.cpu().numpy().astype(np.float64) - old.numpy()
    assert np.all(np.abs(got - want) <= TOL * np.abs(1.5 * size).max(1, keepdims=True) + 2.0 ** -23 * np.abs(old.numpy()))
    none = (idx.numpy() < 0) | (idx.numpy() >= E)
    rows = none.all(1)
    assert rows.any() and torch.equal(acc.cpu()[rows], old[rows])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_against_differences(B, score, renorm):
    """Central differences of the oracle's weights at the chosen ids."""
    T, E, k = 6, 20, 4
    z = inputs.make_router_logits(T, E, 2, "cpu").double().numpy()
    dw = np.random.default_rng(0).standard_normal((T, k)).astype(np.float32)
    idx, _ = og.choose(z, k, score, renorm, scale=1.5)
    shape, p = B.make_shape(T, 256, 128, E, k), B.make_gate_params(score, renorm=renorm, scale=1.5)
    d = B.gate_bwd(shape, p, torch.from_numpy(z).float().to(DEV), torch.from_numpy(idx).int().to(DEV),
                   torch.from_numpy(dw).to(DEV)).cpu().numpy()
    h = 1e-5
    for e in range(E):
        up, dn = z.copy(), z.copy()
        up[:, e] += h
        dn[:, e] -= h
        for t in range(T):
            a = 1.5 * og._weights(up[t], idx[t], score, renorm)
            b = 1.5 * og._weights(dn[t], idx[t], score, renorm)
            assert abs(((a - b) / (2 * h)) @ dw[t] - d[t, e]) <= 1e-5 * 1.5 * np.abs(dw[t]).max() + 1e-9


def test_long_batch_and_rows_behind_it(B):
    """Rows behind the batch stay as they were, for every way a token is handled."""
    for T, E, k, G in ((70001, 64, 4, 8), (3001, 256, 8, 8), (5, 1024, 9, 1), (65, 10, 3, 1)):
        print(f"case behind T={T} E={E}", flush=True)
        z = inputs.make_router_logits(T, E, 1, DEV, 0.5)
        idx = torch.full((T + 4, k), 77, dtype=torch.int32, device=DEV)
        w = torch.full((T + 4, k), 7.5, device=DEV)
        d = torch.full((T + 4, E), 7.5, device=DEV)
        shape, p = B.make_shape(T, 256, 128, E, k), B.make_gate_params("sigmoid", groups=G, groups_kept=max(1, G // 2),
                                                                       group_top=2)
        B.gate(shape, p, z, None, None, idx, w)
        B.gate_bwd(shape, p, z, idx, w, d)
        assert (idx[T:] == 77).all() and (w[T:] == 7.5).all() and (d[T:] == 7.5).all()
        ri, _ = og.choose(z[:200].cpu().numpy(), k, "sigmoid", True, None, G, max(1, G // 2), 2)
        assert np.array_equal(idx[:min(T, 200)].cpu().numpy(), ri)
        again = B.gate(shape, p, z)
        assert torch.equal(again[0], idx[:T]) and torch.equal(again[1], w[:T])


def test_empty_batch(B):
    shape = B.make_shape(0, 256, 128, 8, 2)
    i, w = B.gate(shape, B.make_gate_params(), torch.empty((0, 8), device=DEV))
    assert i.shape == (0, 2) and w.shape == (0, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(41, 60, 4), (30, 256, 8), (19, 600, 3), (9, 1000, 20)])
def test_masked_rows_hold_anything(B, score, renorm, T, E, k):
    """NaN, infinities and the type's lowest in the logits of masked tokens, NaN in their
    gradient: they have no choice, no weight and no gradient, and the others do not notice."""
    print(f"case masked rows T={T} E={E} k={k} {score} {renorm}", flush=True)
    z = inputs.make_router_logits(T, E, 4, DEV, 0.5)
    mask = (torch.arange(T, device=DEV) % 3 != 1).to(torch.uint8)
    out = mask == 0
    wild = z.clone()
    for at, v in ((0, torch.nan), (1, torch.inf), (2, -torch.inf), (3, torch.finfo(torch.float32).min)):
        wild[out, at] = v
    wild[1] = torch.nan
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(3)).to(DEV)
    dw_wild = dw.clone()
    dw_wild[out] = torch.nan
    shape, p = B.make_shape(T, 256, 128, E, k), B.make_gate_params(score, renorm=renorm)
    idx, w = B.gate(shape, p, z, None, mask)
    i2, w2 = B.gate(shape, p, wild, None, mask)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and (idx[out] == -1).all() and not w[out].any()
    d, d2 = B.gate_bwd(shape, p, z, idx, dw), B.gate_bwd(shape, p, wild, idx, dw_wild)
    assert torch.equal(d, d2) and not d2[out].any() and torch.isfinite(d2).all()
    acc = torch.full((T, E), 2.0, device=DEV)
    B.gate_bwd(shape, p, wild, idx, dw_wild, acc, accumulate=True)
    assert (acc[out] == 2).all() and torch.isfinite(acc).all()


def test_offsets_past_32_bits(B):
    """Logits of more than 2^31 elements: tokens at the ends and round the border against the oracle."""
    T, E, k = 2_200_001, 1024, 3
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    print("case gate past 32 bits", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    z = torch.empty((T, E), device=DEV)
    for at in range(0, T, 200_000):
        z[at:at + 200_000] = torch.randn(z[at:at + 200_000].shape, generator=g, device=DEV)
    border = (1 << 31) // E
    rows = torch.tensor([0, 1, border // 2, border - 1, border, border + 1, T - 2, T - 1], device=DEV)
    shape = B.make_shape(T, 256, 128, E, k)
    for score, renorm in (("sigmoid", True), ("softmax", False)):
        p, b = B.make_gate_params(score, renorm=renorm), _bias(E, 3, 0.2 if score == "sigmoid" else 0.5 / E)
        idx, w = B.gate(shape, p, z, b)
        zr = z[rows].cpu().numpy()
        ri, rw = og.choose(zr, k, score, renorm, b.cpu().numpy())
        assert np.array_equal(idx[rows].cpu().numpy(), ri)
        assert np.all(np.abs(w[rows].cpu().numpy() - rw) <= TOL * rw.max(1, keepdims=True))
        dw = torch.randn((T, k), generator=g, device=DEV)
        d = B.gate_bwd(shape, p, z, idx, dw)
        _compare_bwd(d[rows].cpu().numpy(), og.choose_backward(zr, ri, dw[rows].cpu().numpy(), score, renorm),
                     dw[rows].cpu().numpy(), 1.0)
        del d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,L,top", [(128, 8, 1, 1, 1), (256, 8, 8, 4, 2), (60, 4, 1, 1, 1), (512, 15, 1, 1, 1), (512, 16, 1, 1, 1),
                                         (1000, 6, 1, 1, 1), (16, 1, 1, 1, 1), (16, 15, 1, 1, 1), (16, 16, 1, 1, 1),
                                         (256, 8, 8, 2, 1)])
def test_close_pairs_among_spread_scores(B, score, E, k, G, L, top):
    """Well spread rows in which two, three or more of the best k + 3 are equal or a unit or two
    apart, inside the choice, across its end and behind it; biases of few values, so that
    some such pairs stay close and some do not."""
    T = 600
    r = np.random.default_rng(E + k)
    z = (1.5 * r.standard_normal((T, E))).astype(np.float32)
    order = np.argsort(-z, axis=1)
    for t in range(T):
        best = order[t, :min(E, k + 3)]
        n = len(best)
        for _ in range(r.integers(1, 4)):
            at, size = r.integers(0, n), r.integers(2, 5)
            run = best[at:at + size]
            v = z[t, run[0]]
            for e in run[1:]:
                z[t, e] = v
                for _ in range(r.integers(0, 3)):
                    z[t, e] = np.nextafter(z[t, e], np.float32(-10 if r.random() < 0.5 else 10))
    z = torch.from_numpy(z).to(DEV)
    coarse = (torch.arange(E, device=DEV) % 3).float() * 0.03125
    _check(B, z, k, score, True, None, G, L, top)
    _check(B, z, k, score, True, torch.zeros(E, device=DEV), G, L, top)
    _check(B, z, k, score, False, coarse, G, L, top)
    _check(B, z, k, score, True, coarse + _bias(E, 1, 1e-7), G, L, top)
