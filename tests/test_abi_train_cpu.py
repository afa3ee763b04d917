"""Host-side refusals of the balance and orthogonalisation entry points: every
call here is refused, or answered, before anything reaches the GPU."""
import ctypes
import math
import os

import pytest
import torch

from tests.helpers import LIB

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")
P = 1 << 20  # an aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def B():
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


def _call(B, name, shape, *args):
    return getattr(B.lib(), name)(ctypes.byref(shape), *args)


def _balance(B, s, S=1, n=1 << 40, **kw):
    a = dict(logits=P, idx=P, off=P, mask=P, loss=P, counts=P, seq_counts=P, seq_probs=P, seq_scale=P, ws=P)
    a.update(kw)
    return _call(B, "moe_balance", s, a["logits"], a["idx"], a["off"], S, a["mask"], a["loss"], a["counts"],
                 a["seq_counts"], a["seq_probs"], a["seq_scale"], a["ws"], n, None)


def test_balance_refusals(B):
    s = B.make_shape(64, 256, 128, 8, 2)
    need = B.moe_balance_scratch_bytes(s, 3)
    assert need > 0
    for name in ("logits", "idx", "loss", "counts", "seq_counts", "seq_probs", "seq_scale", "ws"):
        assert _balance(B, s, **{name: None}) == 1, name
    for name in ("logits", "idx", "off", "loss", "counts", "seq_counts", "seq_probs", "seq_scale"):
        assert _balance(B, s, **{name: P + 2}) == 3, name
    assert _balance(B, s, n=need - 1, S=3) == 6
    assert _balance(B, s, S=0) == 2 and _balance(B, s, S=-1) == 2
    assert _balance(B, s, S=(1 << 20) + 1) == 2
    assert _balance(B, s, S=2, off=None) == 1          # several sequences need their bounds
    assert _balance(B, B.make_shape(64, 256, 128, 8, 9)) == 2
    assert _balance(B, B.make_shape(64, 256, 128, 1024, 2), S=1 << 19) == 2   # S * E
    assert B.moe_balance_scratch_bytes(s, 0) == 0
    assert B.moe_balance_scratch_bytes(B.make_shape(64, 256, 128, 8, 9), 1) == 0


def _balance_bwd(B, s, S=1, **kw):
    a = dict(logits=P, idx=P, w=P, dw=P, off=P, mask=P, seq_counts=P, seq_scale=P, d_loss=P, d_logits=P)
    a.update(kw)
    return _call(B, "moe_balance_bwd", s, a["logits"], a["idx"], a["w"], a["dw"], 1, a["off"], S, a["mask"],
                 a["seq_counts"], a["seq_scale"], a["d_loss"], a["d_logits"], None)


def test_balance_bwd_refusals(B):
    s = B.make_shape(64, 256, 128, 8, 2)
    for name in ("logits", "seq_counts", "seq_scale", "d_loss", "d_logits", "idx", "w"):
        assert _balance_bwd(B, s, **{name: None}) == 1, name
    for name in ("logits", "idx", "w", "dw", "off", "seq_counts", "seq_scale", "d_loss", "d_logits"):
        assert _balance_bwd(B, s, **{name: P + 1}) == 3, name
    assert _balance_bwd(B, s, S=0) == 2 and _balance_bwd(B, s, S=4, off=None) == 1
    assert _balance_bwd(B, B.make_shape(0, 256, 128, 8, 2), logits=None) == 0   # nothing to do


BAD_ORTHO = [(dict(E=-1), 2), (dict(R=0), 2), (dict(C=0), 2), (dict(R=16385), 2), (dict(C=16385), 2),
             (dict(E=1 << 20, R=1024, C=1024), 2), (dict(steps=0), 2), (dict(steps=33), 2),
             (dict(grad=2), 4), (dict(coeffs=(math.nan, 0, 0)), 2), (dict(coeffs=(1, math.inf, 0)), 2),
             (dict(eps=-1.0), 2), (dict(eps=math.inf), 2)]


@pytest.mark.parametrize("kw,status", BAD_ORTHO)
def test_ortho_shape_refusals(B, kw, status):
    a = dict(E=2, R=64, C=64)
    a.update(kw)
    s = B.make_ortho_shape(**a)
    with pytest.raises(B.MoEError) as ei:
        B.moe_ortho_workspace_size(s)
    assert ei.value.status == status
    assert _call(B, "moe_orthogonalize", s, P, P, P, 1 << 40, None) == status
    s2 = B.make_ortho_shape(2, 64, 64)
    s2.reserved = 1
    assert _call(B, "moe_orthogonalize", s2, P, P, P, 1 << 40, None) == 2


def test_orthogonalize_refusals(B):
    s = B.make_ortho_shape(2, 100, 64)
    need = B.moe_ortho_workspace_size(s)
    f = lambda G=P, U=P, ws=P, n=1 << 40: _call(B, "moe_orthogonalize", s, G, U, ws, n, None)  # noqa: E731
    assert f(G=None) == 1 and f(U=None) == 1 and f(ws=None) == 1
    assert f(G=P + 8) == 3 and f(U=P + 8) == 3 and f(ws=P + 8) == 3
    assert f(n=need - 1) == 6
    assert _call(B, "moe_orthogonalize", B.make_ortho_shape(0, 100, 64), None, None, None, 0, None) == 0
    assert B.lib().moe_orthogonalize(None, P, P, P, 1 << 40, None) == 1


def test_muon_step_refusals(B):
    s = B.make_ortho_shape(2, 100, 64)
    need = B.moe_ortho_workspace_size(s)

    def f(grad=P, mom=P, W=P, master=P, ws=P, n=1 << 40, **kw):
        a = dict(lr=0.1, mu=0.9, weight_decay=0.0, scale=1.0, nesterov=1, reserved=0)
        a.update(kw)
        p = B.moe_muon_params(**a)
        return _call(B, "moe_muon_step", s, ctypes.byref(p), grad, mom, W, master, ws, n, None)

    for name in ("grad", "mom", "W", "ws"):
        assert f(**{name: None}) == 1, name
    for name in ("grad", "mom", "W", "master", "ws"):
        assert f(**{name: P + 4}) == 3, name
    assert f(n=need - 1) == 6
    for kw in (dict(lr=math.nan), dict(mu=1.0), dict(mu=-0.1), dict(mu=math.nan), dict(weight_decay=math.inf),
               dict(scale=math.nan), dict(reserved=1)):
        assert f(**kw) == 2, kw
    assert _call(B, "moe_muon_step", s, None, P, P, P, None, P, 1 << 40, None) == 1


def test_workspace_is_bounded(B):
    """The scratch holds a group of matrices: it does not grow with E forever."""
    a = B.moe_ortho_workspace_size(B.make_ortho_shape(1, 1536, 4096))
    b = B.moe_ortho_workspace_size(B.make_ortho_shape(10 ** 4, 1536, 4096))
    c = B.moe_ortho_workspace_size(B.make_ortho_shape(10 ** 5, 1536, 4096))
    assert a < b == c < (6 << 30)


def test_binding_checks_tensors(B):
    s = B.make_ortho_shape(2, 16, 8)
    G = torch.zeros((2, 16, 8), dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)
    for bad in (G.float(), G.transpose(1, 2), G[:1], G):   # type, strides, size, device
        with pytest.raises(B.MoEError) as ei:
            B.moe_orthogonalize(s, bad, G, ws, stream=0)
        assert ei.value.status == 2
    with pytest.raises(B.MoEError) as ei:
        B.moe_muon_step(s, B.moe_muon_params(0.1, 0.9, 0.0, 1.0, 0, 0), G, G, G, None, ws, stream=0)
    assert ei.value.status == 2
    r = B.make_shape(4, 256, 128, 8, 2)
    z = torch.zeros((4, 8))
    with pytest.raises(B.MoEError) as ei:
        B.moe_balance(r, z.double(), None, None, 1, None, z, z, z, z, z, ws, stream=0)
    assert ei.value.status == 2
    with pytest.raises(B.MoEError) as ei:
        B.moe_balance_bwd(r, z[:, ::2], None, None, None, True, None, 1, None, None, None, None, z, stream=0)
    assert ei.value.status == 2
