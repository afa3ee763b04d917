"""Pins of the gate, dense-product and AdamW oracles: values worked out by hand,
torch's own operations in float64, and central differences."""
import numpy as np
import torch

from oracle import moe_adamw as oa
from oracle import moe_gate as og
from oracle import moe_linear as ol
from oracle import moe_router as rt


def test_choice_without_extras_is_the_routers():
    z = np.random.default_rng(0).standard_normal((50, 20)).astype(np.float32)
    for renorm in (True, False):
        i, w = og.choose(z, 4, "softmax", renorm)
        ri, rw = rt.route(z, 4, renorm)
        assert np.array_equal(i, ri) and np.allclose(w, rw, rtol=1e-14)
        dw = np.random.default_rng(1).standard_normal((50, 4))
        assert np.allclose(og.choose_backward(z, i, dw, "softmax", renorm), rt.route_backward(z, i, dw, renorm), atol=1e-14)


def test_choice_by_hand():
    """Sigmoid scores 0.5, 0.5, 0.75, 0.25 of logits 0, 0, ln 3, -ln 3."""
    z = np.array([[0.0, 0.0, np.log(3.0), -np.log(3.0)]])
    i, w = og.choose(z, 2, "sigmoid", False)
    assert i.tolist() == [[2, 0]] and np.allclose(w, [[0.75, 0.5]])
    i, w = og.choose(z, 2, "sigmoid", True, bias=[0, 0, 0, 1.0], scale=2.0)
    assert i.tolist() == [[3, 2]] and np.allclose(w, [[0.5, 1.5]])
    # groups {0, 1} and {2, 3}: sums of two 1.0 and 1.0 (the lower group), largest 0.5 and 0.75
    assert og.choose(z, 1, "sigmoid", True, groups=2, kept=1, top=2)[0].tolist() == [[0]]
    assert og.choose(z, 1, "sigmoid", True, groups=2, kept=1, top=1)[0].tolist() == [[2]]
    z[0, :2] = -np.inf
    i, w = og.choose(z, 3, "sigmoid", True, groups=2, kept=2, top=2)
    assert i.tolist() == [[2, 3, -1]] and np.allclose(w, [[0.75, 0.25, 0.0]])
    assert og.choose(z, 3, mask=[0])[0].tolist() == [[-1, -1, -1]]
    assert np.isnan(og.choose([[np.nan, 1.0]], 1)[1]).all()


def test_weights_of_scores_that_underflow():
    i, w = og.choose([[-2000.0, -2000.0 + np.log(3.0)]], 2, "sigmoid", True)
    assert i.tolist() == [[1, 0]] and np.allclose(w, [[0.75, 0.25]], rtol=1e-12)


def test_gate_gradient_against_differences():
    g = np.random.default_rng(3)
    z, dw = g.standard_normal((3, 9)), g.standard_normal((3, 4))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx, _ = og.choose(z, 4, score, renorm)
            d = og.choose_backward(z, idx, dw, score, renorm, 1.5)
            for e in range(9):
                h = np.zeros_like(z)
                h[:, e] = 1e-6
                for t in range(3):
                    f = lambda y: 1.5 * og._weights(y[t], idx[t], score, renorm) @ dw[t]  # noqa: E731
                    assert abs((f(z + h) - f(z - h)) / 2e-6 - d[t, e]) < 1e-8


def test_dense_products_against_autograd():
    g = torch.Generator().manual_seed(0)
    for act, f in (("none", lambda p: p), ("relu", torch.relu), ("silu", torch.nn.functional.silu),
                   ("gelu", lambda p: torch.nn.functional.gelu(p, approximate="tanh")),
                   ("swiglu", lambda p: torch.nn.functional.silu(p[:, :5]) * p[:, 5:])):
        R = 10 if act == "swiglu" else 5
        X, W, b = (torch.randn(s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((7, 6), (R, 6), (R,)))
        res, dY = (torch.randn((7, 5), generator=g, dtype=torch.float64) for _ in range(2))
        Pt = X @ W.t() + b
        Yt = f(Pt) + res
        n = lambda t: t.detach().numpy()  # noqa: E731
        Y, P = ol.linear(n(X), n(W), n(b), n(res), act)
        assert np.allclose(Y, n(Yt), rtol=1e-12) and np.allclose(P, n(Pt), rtol=1e-12)
        Yt.backward(dY)
        dX, dW, db, _ = ol.linear_backward(n(dY), n(X), n(W), P, act)
        for a, t in ((dX, X), (dW, W), (db, b)):
            assert np.allclose(a, t.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_adamw_against_torch():
    g = torch.Generator().manual_seed(1)
    w = torch.randn(50, generator=g, dtype=torch.float64)
    p = w.clone().requires_grad_(True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    a, m, v = w.numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 5):
        p.grad = torch.randn(50, generator=g, dtype=torch.float64)
        opt.step()
        a, m, v = oa.step(a, p.grad.numpy(), m, v, lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-6, weight_decay=0.1, t=t)
        assert np.allclose(a, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_codes_are_e4m3():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, oa.E4M3, equal_nan=True)
    x = np.random.default_rng(0).standard_normal(1000).astype(np.float32) * 10.0 ** np.repeat(np.arange(-4, 4), 125)
    codes, scale = oa.encode(x)
    s = 2.0 ** (scale.astype(np.float64) - 127)
    for b in range(8):
        v = x[b * 128:(b + 1) * 128].astype(np.float64)
        assert 448 * s[b] >= np.abs(v).max() > 224 * s[b]
        want = torch.from_numpy(v / s[b]).float().to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(oa.E4M3[codes[b * 128:(b + 1) * 128]], want)
    c, s = oa.encode([0.0, 1e-9, 448.0, np.nan], keep=True)
    assert c.tolist() == [0, 1, 0x7E, 0x7F] and s.tolist() == [127]
    assert oa.encode([449.0])[1].tolist() == [128] and oa.encode(np.zeros(5))[1].tolist() == [127]
