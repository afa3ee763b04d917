"""The routing balance on finite logits of any magnitude, to the ends of fp32,
as fully masked rows hold them (a sentinel in place of -inf), against the
float64 oracle and against moe_route_bwd.

Bounds. In rows of such magnitude logits are equal or so far apart that the
softmax is 0 or 1 / ties; ordinary rows are as in test_gpu_balance.py, whose
TOL = 1e-5 holds. A gradient is compared row by row: it is a difference of
terms as large as the row's balance factors B, its d_topk_w and its z-term,
so it may be off by TOL times their sum. loss[1] is fp32: what passes its
range is inf."""
import math

import numpy as np
import pytest
import torch

from grouped_gemm_02_amd import inputs
from oracle import moe_balance as ob
from tests.helpers import max_rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-5
FMAX = torch.finfo(torch.float32).max
VALUES = [-5e9, 1e10, -1e10, -1e30, 1e30, 2.5e38, FMAX, -FMAX]
SHAPES = [(64, 8, 2, 1), (3000, 24, 3, 3), (40, 300, 4, 2)]   # one workgroup; three launches; two chunks a lane


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _np(t):
    return None if t is None else t.cpu().numpy()


def _batch(T, E, k, S, v):
    """Ordinary rows, and among them rows whose largest logit is v, some masked."""
    z = inputs.make_router_logits(T, E, 11, DEV, skew=0.6)
    z[5] = v                                  # every expert, as a mask of sentinels leaves it
    z[6] = v                                  # the same, masked out below
    z[7] = -FMAX                              # v on three experts, the rest at the lowest value
    z[7, 1:4] = v
    z[8] = z[7]                               # masked out below
    if v > 0:
        z[9, E - 1] = v                       # one far above ordinary ones
    _, idx = torch.topk(z, k, dim=1)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[[6, 8, 20]] = 0
    off = None if S == 1 else torch.tensor([0] + [T * (q + 1) // S for q in range(S)], dtype=torch.int32, device=DEV)
    return z, idx.to(torch.int32).contiguous(), off, mask


@pytest.mark.parametrize("T,E,k,S", SHAPES)
@pytest.mark.parametrize("v", VALUES)
def test_losses_of_large_finite_rows(B, T, E, k, S, v):
    print(f"case balance range T={T} E={E} S={S} v={v:g}", flush=True)
    z, idx, off, mask = _batch(T, E, k, S, v)
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), S)
    B.balance(buf, z, idx, off, mask)
    torch.cuda.synchronize()
    ref = ob.balance(_np(z), _np(idx), _np(off), _np(mask))
    assert np.array_equal(_np(buf.seq_counts), ref["seq_counts"])
    for name in ("seq_probs", "seq_scale"):
        assert max_rel_err(_np(getattr(buf, name)), ref[name]) <= TOL, name
    got = _np(buf.loss)
    assert abs(got[0] - ref["loss"][0]) <= TOL * ref["loss"][0]
    if ref["loss"][1] > FMAX:
        assert got[1] == math.inf
    else:
        assert abs(got[1] - ref["loss"][1]) <= TOL * ref["loss"][1]


@pytest.mark.parametrize("T,E,k,S", SHAPES)
@pytest.mark.parametrize("v", VALUES)
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_large_finite_rows(B, T, E, k, S, v, renorm):
    print(f"case balance_bwd range T={T} E={E} S={S} v={v:g} renorm={renorm}", flush=True)
    z, idx, off, mask = _batch(T, E, k, S, v)
    s = B.make_shape(T, 256, 128, E, k)
    w = torch.empty((T, k), device=DEV)
    B.moe_route(s, z, renorm, torch.empty_like(idx), w)
    dw = torch.randn((T, k), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    ref = ob.balance(_np(z), _np(idx), _np(off), _np(mask))
    buf = B.BalanceBuffers.allocate(s, S)
    counts = torch.from_numpy(ref["seq_counts"].astype(np.int32)).to(DEV)
    scale = torch.from_numpy(ref["seq_scale"].astype(np.float32)).to(DEV)
    lse = np.logaddexp.reduce(_np(z).astype(np.float64), axis=1)
    for dl in ((1.0, 0.0), (0.5, 0.01)):
        dl = torch.tensor(dl, device=DEV)
        top = np.abs(dl[0].item() * ref["seq_scale"][:-1, None] * ref["seq_counts"]).max()
        size = top + np.abs(2 * dl[1].item() * ref["seq_scale"][-1] * lse)[:, None]
        for d in (None, dw):
            dz = B.balance_bwd(buf, z, idx, w, d, renorm, dl, off, mask, counts, scale)
            torch.cuda.synchronize()
            want = ob.balance_backward(_np(z), _np(idx), _np(w), _np(d), renorm, _np(dl).astype(np.float64), _np(off),
                                       _np(mask))
            bound = TOL * (size + (0 if d is None else np.abs(_np(d)).sum(1, keepdims=True)))
            assert np.all(np.abs(_np(dz) - want) <= bound), np.argwhere(~(np.abs(_np(dz) - want) <= bound))[:4]
    # without the losses it is moe_route_bwd
    dz, zero = torch.empty_like(z), torch.zeros(2, device=DEV)
    B.moe_route_bwd(s, z, idx, w, dw, renorm, dz)
    alone = B.balance_bwd(buf, z, idx, w, dw, renorm, zero, off, mask, counts, scale)
    assert ((alone - dz).abs() <= TOL * dw.abs().sum(1, keepdim=True)).all().item()


@pytest.mark.parametrize("T,E,k,S", SHAPES)
@pytest.mark.parametrize("v", [2e19, -1e20, 3e20])
def test_squares_past_fp32_whose_mean_is_not(B, T, E, k, S, v):
    """lse^2 of one row leaves fp32, the mean over the tokens does not."""
    print(f"case balance lse^2 T={T} E={E} S={S} v={v:g}", flush=True)
    z, idx, off, mask = _batch(T, E, k, S, 1e10)
    z[7] = v / 4 if T < 1000 else v
    buf = B.BalanceBuffers.allocate(B.make_shape(T, 256, 128, E, k), S)
    B.balance(buf, z, idx, off, mask)
    torch.cuda.synchronize()
    want = ob.balance(_np(z), _np(idx), _np(off), _np(mask))["loss"][1]
    got = buf.loss[1].item()
    assert got == math.inf if want > FMAX else abs(got - want) <= TOL * want
