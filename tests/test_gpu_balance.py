"""GPU parity of the routing balance (moe_balance, moe_balance_bwd) against the
float64 oracle. Counts are equal; floating results within TOL of the largest
value of their tensor. TOL, from the arithmetic (unit u = 2^-24): a
probability is off by the rounding of z - max (20 u for differences up to 20),
exp (2 u), the row sum (at most 4 * 4 + 6 additions) and two more operations,
below 48 u; the sums over a workgroup's tokens add at most 16 + 64 roundings
of positive terms, later sums are in 64 bits: 128 u = 7.6e-6. The backward
takes differences of such values (p (G - <p, G>)), each below its tensor's
largest: the same bound with one more row sum."""
import math

import numpy as np
import pytest
import torch

from grouped_gemm_02_amd import inputs
from oracle import moe_balance as ob
from oracle import moe_router as rt
from tests.helpers import max_rel_err

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


def _poison(buf):
    for t in (buf.loss, buf.counts, buf.seq_counts, buf.seq_probs, buf.seq_scale):
        t.fill_(-77)
    buf.ws.fill_(0xFF)


def _inputs(T, E, k, S, tail, drop, cold, seed):
    z = inputs.make_router_logits(T, E, seed, DEV, skew=0.6)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    if cold:
        z[:, E - cold:] = -math.inf
    _, idx = torch.topk(z, k, dim=1)
    idx = idx.to(torch.int32).contiguous()
    n = T - tail
    cut = torch.sort(torch.randint(0, n + 1, (S - 1,), generator=g, device=DEV)).values
    off = torch.cat([torch.zeros(1, device=DEV), cut, torch.full((1,), n, device=DEV)]).to(torch.int32)
    mask = (torch.rand((T,), generator=g, device=DEV) >= drop).to(torch.uint8) if drop else None
    return z, idx, (off if S > 1 or tail else None), mask


def _np(t):
    return None if t is None else t.cpu().numpy()


CASES = [
    # (T, E, k, S, tail, drop, cold, renorm)
    (1, 1, 1, 1, 0, 0.0, 0, True),
    (1, 8, 2, 1, 0, 0.0, 0, False),
    (64, 8, 2, 1, 0, 0.0, 0, True),
    (33, 16, 1, 1, 0, 0.5, 0, True),          # one chunk and one token
    (500, 17, 3, 7, 11, 0.2, 2, False),       # rows of odd length, a partial last chunk of four
    (1000, 60, 4, 40, 3, 0.2, 2, False),      # several sequences in a chunk
    (257, 64, 64, 3, 0, 0.0, 0, True),        # every expert selected
    (3000, 128, 8, 1, 0, 0.0, 0, True),
    (2049, 129, 8, 5, 100, 0.9, 0, False),
    (777, 256, 8, 2, 0, 0.1, 5, True),
    (300, 500, 70, 3, 1, 0.1, 0, True),       # k beyond the lanes of a row
    (130, 1024, 8, 2, 0, 0.1, 100, False),
    (200, 24, 3, 200, 0, 0.0, 0, True),       # as many sequences as tokens
    (40000, 33, 2, 3, 5, 0.1, 0, True),       # chunks of 64 tokens
    (5000, 40, 3, 2500, 7, 0.1, 0, True),     # more sequences than threads
    (64, 1024, 3, 1, 9, 0.5, 0, True),
    (1024, 64, 4, 1, 13, 0.1, 0, True),       # the most that one workgroup does
    (1025, 64, 4, 1, 13, 0.1, 0, True),
    (32, 1000, 3, 1, 0, 0.1, 7, False),       # one workgroup, all its threads' experts
]


@pytest.mark.parametrize("T,E,k,S,tail,drop,cold,renorm", CASES)
def test_balance_and_gradient_match_oracle(B, T, E, k, S, tail, drop, cold, renorm):
    print(f"case balance T={T} E={E} k={k} S={S} tail={tail} drop={drop} cold={cold} renorm={renorm}", flush=True)
    z, idx, off, mask = _inputs(T, E, k, S, tail, drop, cold, T + E + k)
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), S)
    _poison(buf)
    B.balance(buf, z, idx, off, mask)
    torch.cuda.synchronize()
    ref = ob.balance(_np(z), _np(idx), _np(off), _np(mask))
    assert np.array_equal(_np(buf.counts), ref["counts"])
    assert np.array_equal(_np(buf.seq_counts), ref["seq_counts"])
    for name in ("loss", "seq_probs", "seq_scale"):
        assert max_rel_err(_np(getattr(buf, name)), ref[name]) <= TOL, name
    g = torch.Generator(device=DEV).manual_seed(5)
    dw = torch.randn((T, k), generator=g, device=DEV) * 1e-2
    w = torch.from_numpy(np.take_along_axis(np.exp(rt_log_softmax(_np(z))), _np(idx).astype(np.int64), 1)).float()
    w = (w / w.sum(1, keepdim=True) if renorm else w).to(DEV).contiguous()
    dl = torch.tensor([0.5, 0.01], device=DEV)
    for d in (dw, None):
        dz = torch.full((T, E), -77.0, device=DEV)
        B.balance_bwd(buf, z, idx, w, d, renorm, dl, off, mask, d_logits=dz)
        torch.cuda.synchronize()
        want = ob.balance_backward(_np(z), _np(idx), _np(w), _np(d), renorm, _np(dl).astype(np.float64), _np(off),
                                   _np(mask))
        assert max_rel_err(_np(dz), want) <= TOL, d is None


def rt_log_softmax(z):
    z = z.astype(np.float64)
    m = z.max(1, keepdims=True)
    return z - m - np.log(np.exp(z - m).sum(1, keepdims=True))


def test_gradient_joins_route_bwd(B):
    """With d_loss = 0 the joined backward is moe_route_bwd; with d_topk_w it
    is the sum of the two."""
    T, E, k = 1000, 128, 8
    for renorm in (True, False):
        z = inputs.make_router_logits(T, E, 3, DEV, skew=1.2)
        shape = B.make_shape(T, 256, 128, E, k)
        idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
        w, dz = torch.empty((T, k), device=DEV), torch.empty((T, E), device=DEV)
        B.moe_route(shape, z, renorm, idx, w)
        dw = torch.randn((T, k), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
        B.moe_route_bwd(shape, z, idx, w, dw, renorm, dz)
        buf = B.balance(B.BalanceBuffers.allocate(shape), z, idx)
        zero, one = torch.zeros(2, device=DEV), torch.tensor([3.0, 0.1], device=DEV)
        alone = B.balance_bwd(buf, z, idx, w, dw, renorm, zero)
        loss = B.balance_bwd(buf, z, None, None, None, renorm, one)
        both = B.balance_bwd(buf, z, idx, w, dw, renorm, one)
        torch.cuda.synchronize()
        scale = dz.abs().max().item() + loss.abs().max().item()
        assert (alone - dz).abs().max().item() <= TOL * scale
        assert (both - dz - loss).abs().max().item() <= 2 * TOL * scale


def test_nonfinite_and_dead_rows(B):
    """Rows of -inf, NaN in rows that do not count, ids out of range, one
    expert named twice."""
    T, E, k = 70, 40, 3
    z, idx, _, _ = _inputs(T, E, k, 1, 0, 0.0, 0, 4)
    off = torch.tensor([5, 30, 30, 60], dtype=torch.int32, device=DEV)   # an empty one; head and tail outside
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[10] = 0
    z[12] = -math.inf
    z[:, 7] = -math.inf
    clean = z.clone()
    z[10] = math.nan        # masked
    z[3, 5] = math.nan      # before the first sequence
    z[65] = math.inf        # behind the last
    idx[20, 1] = E
    idx[21, 0] = -1
    idx[22, 2] = idx[22, 0]
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), 3)
    _poison(buf)
    B.balance(buf, z, idx, off, mask)
    torch.cuda.synchronize()
    ref = ob.balance(_np(clean), _np(idx), _np(off), _np(mask))
    assert np.array_equal(_np(buf.seq_counts), ref["seq_counts"]) and np.array_equal(_np(buf.counts), ref["counts"])
    for name in ("loss", "seq_probs", "seq_scale"):
        assert max_rel_err(_np(getattr(buf, name)), ref[name]) <= TOL, name
    dl = torch.tensor([1.0, 0.1], device=DEV)
    dz = B.balance_bwd(buf, z, None, None, None, True, dl, off, mask)
    want = ob.balance_backward(_np(clean), _np(idx), None, None, True, _np(dl).astype(np.float64), _np(off), _np(mask))
    got, rows = _np(dz), np.ones(T, dtype=bool)
    rows[[3, 10, 65]] = False
    assert max_rel_err(got[rows], want[rows]) <= TOL
    assert not got[12].any()
    # a NaN in a live row makes its sequence's losses NaN
    z[40, 2] = math.nan
    B.balance(buf, z, idx, off, mask)
    assert torch.isnan(buf.loss).all().item()
    assert torch.isnan(buf.seq_probs[2]).any().item() and torch.isfinite(buf.seq_probs[0]).all().item()


def test_gradient_of_dead_rows_with_nonfinite_logits(B):
    """Rows outside the losses take nothing from their logits: their gradient is
    0, or that of the renormalised weights, whatever the logits hold."""
    T, E, k = 70, 40, 3
    z, idx, _, _ = _inputs(T, E, k, 1, 0, 0.0, 0, 4)
    off = torch.tensor([5, 30, 30, 60], dtype=torch.int32, device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[10] = 0
    s = B.make_shape(T, 256, 128, E, k)
    w = torch.empty((T, k), device=DEV)
    B.moe_route(s, z, True, idx, w)
    clean = z.clone()
    z[10], z[3, 5], z[65], z[62] = math.nan, math.nan, math.inf, -math.inf
    dead = [10, 3, 65, 62]
    buf = B.BalanceBuffers.allocate(s, 3)
    B.balance(buf, z, idx, off, mask)
    dl = torch.tensor([1.0, 0.1], device=DEV)
    dw = torch.randn((T, k), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    for d in (None, dw):
        dz = _np(B.balance_bwd(buf, z, idx, w, d, True, dl, off, mask))
        want = ob.balance_backward(_np(clean), _np(idx), _np(w), _np(d), True, _np(dl).astype(np.float64), _np(off),
                                   _np(mask))
        assert max_rel_err(dz, want) <= TOL
        assert d is not None or not dz[dead].any()


def test_nothing_live_and_no_tokens(B):
    E, k = 24, 2
    z, idx, _, _ = _inputs(50, E, k, 1, 0, 0.0, 0, 6)
    for T, off, mask in ((50, None, torch.zeros(50, dtype=torch.uint8, device=DEV)),
                         (50, torch.tensor([20, 20, 20], dtype=torch.int32, device=DEV), None),
                         (0, torch.tensor([0, 0, 0], dtype=torch.int32, device=DEV), None)):
        S = 1 if off is None else off.numel() - 1
        buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), S)
        _poison(buf)
        B.balance(buf, z[:T], idx[:T], off, mask)
        for t in (buf.loss, buf.counts, buf.seq_counts, buf.seq_probs, buf.seq_scale):
            assert not t.any().item()
        if T:
            dz = B.balance_bwd(buf, z, idx, None, None, True, torch.ones(2, device=DEV), off, mask)
            assert not dz.any().item()


def test_rows_at_any_4_byte_address_and_repeatable(B):
    """Logits and gradients that start 4 bytes into a buffer; two runs agree
    bit for bit."""
    T, E, k = 900, 61, 4
    z, idx, off, mask = _inputs(T, E, k, 4, 7, 0.2, 0, 8)
    flat = torch.empty(T * E + 3, device=DEV)
    flat[1:1 + T * E] = z.reshape(-1)
    zu = flat[1:1 + T * E].view(T, E)
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), 4)
    B.balance(buf, z, idx, off, mask)
    first = [t.clone() for t in (buf.loss, buf.counts, buf.seq_counts, buf.seq_probs, buf.seq_scale)]
    _poison(buf)
    B.balance(buf, zu, idx, off, mask)
    for a, b in zip(first, (buf.loss, buf.counts, buf.seq_counts, buf.seq_probs, buf.seq_scale)):
        assert torch.equal(a, b)
    dl = torch.tensor([1.0, 0.1], device=DEV)
    a = B.balance_bwd(buf, z, None, None, None, True, dl, off, mask)
    out = torch.full((T * E + 3,), -5.0, device=DEV)
    B.balance_bwd(buf, zu, None, None, None, True, dl, off, mask, d_logits=out[1:1 + T * E].view(T, E))
    assert torch.equal(a, out[1:1 + T * E].view(T, E))
    assert out[0].item() == -5.0 and (out[1 + T * E:] == -5.0).all().item()
