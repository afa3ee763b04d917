"""GPU parity of moe_adamw_step against the float64 oracle.

fp32 moments: m and v are sums of two products of numbers rounded once to fp32 (the betas
and their complements too): 4 roundings, 2^-22 of the larger term. The update is m times a
rounded step, a reciprocal and a root of one unit each, products and a sum: at most 12
roundings, 12 * 2^-24 < 1e-6 of the update; w (1 - lr wd) - update adds two of w. A bf16
parameter is rounded once more: 2^-8 of itself. Moments in 8 bits: the step uses the fresh
ones, so w has the same bounds; codes are compared through their values: each is a nearest
code of a number that is off by 2^-22, so it is within half a step (2^-4 of the value, or
2^-10 of the scale below the normal range) and a little."""
import numpy as np
import pytest
import torch

from oracle import moe_adamw as oa

pytestmark = pytest.mark.gpu
DEV = "cuda"
H = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tensors(sizes, param, grad, seed, shift=0):
    """Parameters and gradients; with `shift` views that begin that many elements into a buffer."""
    g = torch.Generator().manual_seed(seed)
    mk = lambda n, s, dt: (s * torch.randn(n + shift, generator=g)).to(dt).to(DEV)[shift:]  # noqa: E731
    return ([mk(n, 0.05, TYPES[param]) for n in sizes],
            [mk(n, 10.0 ** -(i % 5), TYPES[grad]) for i, n in enumerate(sizes)])


def _n(t):
    return t.double().cpu().numpy().reshape(-1)


def _check_w(got, want, old, dtype):
    upd = np.abs(want - old) + 1e-30
    tol = 2e-6 * upd + 3 * 2.0 ** -24 * (np.abs(old) + np.abs(want))
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))


def _near_code(codes, scale, want, keep):
    """Every held value is the nearest, or next to a border."""
    v = oa.decode(codes, scale)
    s = np.repeat(2.0 ** (scale.astype(np.float64) - 127), 128)[:len(codes)]
    off = np.abs(v - want)
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s) * (1 + 1e-5)
    if keep:
        tol = np.where((codes == 1), np.maximum(tol, 2.0 ** -9 * s), tol)
        assert np.all(codes[want > 0] != 0)
    assert np.all(off <= tol), float(np.max(off / tol))
    assert np.array_equal(scale, oa.encode(want, keep)[1])


SIZES = [[1], [7, 1, 128, 129], [8192, 8193, 100, 3], [20000, 65, 127, 1, 1000], [1 << 17]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: str(sum(s)))
@pytest.mark.parametrize("param,grad,master", [("bf16", "bf16", False), ("bf16", "f32", True), ("bf16", "bf16", True),
                                               ("f32", "f32", False), ("f32", "bf16", False), ("bf16", "f32", False)])
@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps_match_oracle(B, sizes, param, grad, master, state, shift):
    """Three steps, each against the oracle from the state the kernel left."""
    print(f"case adamw {sizes} {param} {grad} master={master} {state} shift={shift}", flush=True)
    P, G = _tensors(sizes, param, grad, len(sizes), shift)
    n = len(sizes)
    mul, dec = [1.0 + 0.5 * (i % 3) for i in range(n)], [float(i % 2) for i in range(n)]
    buf = B.AdamWBuffers.allocate(P, state=state, master=master, lr_mul=mul, decay_mul=dec)
    clip = torch.tensor([0.37], device=DEV)
    for t in range(1, 4):
        old = [(_n(buf.master[i]) if master else _n(P[i])) for i in range(n)]
        if state == "f32":
            mv = [(_n(buf.m[i]), _n(buf.v[i])) for i in range(n)]
        else:
            mv = [(oa.decode(buf.m[i].cpu().numpy(), buf.m_scale[i].cpu().numpy()),
                   oa.decode(buf.v[i].cpu().numpy(), buf.v_scale[i].cpu().numpy()) ** 2) for i in range(n)]
        B.adamw_step(buf, G, step=t, grad_scale=clip if t > 1 else None, **H)
        for i in range(n):
            h = dict(H, lr=H["lr"] * mul[i], weight_decay=H["weight_decay"] * dec[i])
            w, m, v = oa.step(old[i], _n(G[i]), *mv[i], t=t, grad_scale=float(clip.cpu()[0]) if t > 1 else 1.0, **h)
            if master:
                _check_w(_n(buf.master[i]), w, old[i], torch.float32)
                assert torch.equal(P[i].view(-1), buf.master[i].to(torch.bfloat16))
            else:
                _check_w(_n(P[i]), w, old[i], P[i].dtype)
            if state == "f32":
                a, b = np.abs(mv[i][0]), np.abs(_n(G[i]))
                assert np.all(np.abs(_n(buf.m[i]) - m) <= 2.0 ** -22 * (a + b))
                assert np.all(np.abs(_n(buf.v[i]) - v) <= 2.0 ** -21 * v + 1e-38)
            else:
                _near_code(buf.m[i].cpu().numpy(), buf.m_scale[i].cpu().numpy(), m, False)
                _near_code(buf.v[i].cpu().numpy(), buf.v_scale[i].cpu().numpy(), np.sqrt(v), True)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_many_tensors(B, state):
    """More tensors than one launch takes, some without elements, some passed over."""
    sizes = [(37 * i) % 400 for i in range(131)]
    P, G = _tensors(sizes, "f32", "f32", 3)
    master = None
    buf = B.AdamWBuffers.allocate(P, state=state, master=False)
    old = [p.clone() for p in P]
    grads = [None if i % 10 == 4 else g for i, g in enumerate(G)]
    B.adamw_step(buf, grads, step=1, **H)
    for i, s in enumerate(sizes):
        if grads[i] is None:
            assert torch.equal(P[i], old[i]) and not buf.m[i].any()
        elif s:
            _check_w(_n(P[i]), oa.step(_n(old[i]), _n(G[i]), 0 * _n(G[i]), 0 * _n(G[i]), t=1, **H)[0], _n(old[i]),
                     torch.float32)
    # masters on some of the tensors only
    P, G = _tensors(sizes, "bf16", "bf16", 4)
    master = [p.float().clone() if i % 3 else None for i, p in enumerate(P)]
    z = lambda dt: [torch.zeros(s, dtype=dt, device=DEV) for s in sizes]  # noqa: E731
    b = lambda: [torch.zeros(-(-s // 128), dtype=torch.uint8, device=DEV) for s in sizes]  # noqa: E731
    buf = (B.AdamWBuffers(P, z(torch.float32), z(torch.float32), None, None, master) if state == "f32" else
           B.AdamWBuffers(P, z(torch.uint8), z(torch.uint8), b(), b(), master))
    old = [p.clone() for p in P]
    B.adamw_step(buf, G, step=1, **H)
    for i, s in enumerate(sizes):
        if s:
            w = oa.step(_n(old[i]), _n(G[i]), 0 * _n(G[i]), 0 * _n(G[i]), t=1, **H)[0]
            _check_w(_n(P[i] if master[i] is None else master[i]), w, _n(old[i]),
                     torch.bfloat16 if master[i] is None else torch.float32)


def _one(B, state, n, param="f32"):
    P, G = _tensors([n], param, "f32", 5)
    buf = B.AdamWBuffers.allocate(P, state=state)
    return P[0], G[0], buf


@pytest.mark.parametrize("state", ["f32", "8bit"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_scale_that_is_not_finite_changes_nothing(B, state, bad):
    p, g, buf = _one(B, state, 3000)
    B.adamw_step(buf, [g], step=1, **H)
    keep = [t.clone() for t in (p, buf.m[0], buf.v[0])]
    B.adamw_step(buf, [g], step=2, grad_scale=torch.tensor([bad], device=DEV), **H)
    hy = torch.tensor([1e-3, 0.19, 0.1, bad], device=DEV)
    B.adamw_step(buf, [g], step=2, hyper=hy, **H)
    for a, b in zip((p, buf.m[0], buf.v[0]), keep):
        assert torch.equal(a, b)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_values_from_the_device(B, state):
    p, g, buf = _one(B, state, 5000)
    q, h, ref = _one(B, state, 5000)
    for t in (1, 2, 3):
        B.adamw_step(ref, [h], step=t, grad_scale=torch.tensor([0.5], device=DEV), **H)
        hy = torch.tensor([H["lr"], 1 - H["beta1"] ** t, 1 - H["beta2"] ** t, 0.5], device=DEV)
        B.adamw_step(buf, [g], step=1, hyper=hy, **dict(H, lr=7.0))
    # the corrections pass through fp32: a unit or two of the update
    assert torch.allclose(p, q, rtol=1e-6, atol=3 * H["lr"] * 1e-6)
    assert torch.equal(buf.m[0], ref.m[0])


def test_eight_bits_at_their_ends(B):
    """Blocks of zeros, of one value, of tiny and huge ones; gradients that are not finite
    leave NaN in their elements and the others' codes as they should be."""
    n = 128 * 9 + 5
    g = torch.zeros(n)
    g[128:256] = 448.0 * 10
    g[256:384] = 449.0 * 10
    g[384:512] = torch.linspace(1e-30, 1e-28, 128)
    g[512:640] = torch.linspace(-1e15, 1e15, 128)
    g[640:768] = torch.logspace(-20, 3, 128)
    g[768:896] = 1.0
    g[800], g[801], g[802] = torch.nan, torch.inf, -torch.inf
    g[896:1024] = -2.0 ** -10
    g[1152:] = 3.0
    G = g.to(DEV)
    p = torch.zeros(n, device=DEV)
    buf = B.AdamWBuffers.allocate([p], state="8bit")
    B.adamw_step(buf, [G], lr=1e-3, beta1=0.9, beta2=0.95, step=1)
    x = g.double().numpy()
    f = np.isfinite(x)
    _, m, v = oa.step(0 * x, x, 0 * x, 0 * x, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, t=1)
    mc, ms, vc, vs = (t.cpu().numpy() for t in (buf.m[0], buf.m_scale[0], buf.v[0], buf.v_scale[0]))
    assert np.all((mc[~f] & 0x7F) == 0x7F) and np.all(vc[~f] == 0x7F)
    assert mc[:128].max() == 0 and vc[:128].max() == 0 and ms[0] == 127 and vs[0] == 127
    # v of 1e-30 squared is below fp32's range: held as 0 (m is not)
    small = np.zeros(n, bool)
    small[384:512] = True
    small |= (np.abs(x) < 1e-18)
    # zeros in the place of what is not finite: the block's scale comes from the others
    _near_code(np.where(f, mc, 0), ms, np.where(f, m, 0.0), False)
    r = np.sqrt(np.where(f, v, 0.0))
    dec = oa.decode(np.where(f, vc, 0), vs)
    ok = f & ~small
    s = np.repeat(2.0 ** (vs.astype(np.float64) - 127), 128)[:n]
    tol = np.maximum(2.0 ** -4 * r, 2.0 ** -10 * s) * (1 + 1e-5)
    tol = np.where(vc == 1, np.maximum(tol, 2.0 ** -9 * s), tol)
    assert np.all(np.abs(dec - r)[ok] <= tol[ok])
    assert np.all(vc[ok & (r > 0)] != 0)
    assert torch.isnan(p.cpu()[~torch.from_numpy(f)]).all() and torch.isfinite(p.cpu()[torch.from_numpy(f)]).all()


def test_sides_of_a_tensor_are_left_alone(B):
    """Elements before and behind a view, and codes behind a tensor's end."""
    for state in ("f32", "8bit"):
        for n in (1, 5, 127, 2049):
            whole = torch.full((n + 20,), 3.0, dtype=torch.bfloat16, device=DEV)
            g = torch.ones(n, dtype=torch.bfloat16, device=DEV)
            dt = torch.float32 if state == "f32" else torch.uint8
            m, v = torch.full((n + 20,), 1, dtype=dt, device=DEV), torch.full((n + 20,), 1, dtype=dt, device=DEV)
            k = -(-n // 128)
            ms, vs = (torch.full((k + 2,), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
            buf = B.AdamWBuffers([whole[7:7 + n]], [m[:n]], [v[:n]], None if state == "f32" else [ms[:k]],
                                 None if state == "f32" else [vs[:k]])
            B.adamw_step(buf, [g], step=3, **H)
            assert (whole[:7] == 3).all() and (whole[7 + n:] == 3).all()
            # moments of 1 (8-bit: code 1 is 2^-9 and scale 1) and a gradient of 1; an update below
            # half of bf16's spacing at 3 (2^-7) leaves the rounded parameter where it is
            x = np.ones(n) if state == "f32" else np.full(n, 2.0 ** -9)
            want = oa.step(np.full(n, 3.0), np.ones(n), x, x if state == "f32" else x * x, t=3, **H)[0]
            _check_w(_n(whole[7:7 + n]), want, np.full(n, 3.0), torch.bfloat16)
            assert (m[n:] == 1).all() and (v[n:] == 1).all() and (ms[k:] == 127).all() and (vs[k:] == 127).all()


def test_captured_steps_follow_the_device_values(B):
    p, g, buf = _one(B, "8bit", 10000, "bf16")
    q, h, ref = _one(B, "8bit", 10000, "bf16")
    hy = torch.tensor([0.0, 1.0, 1.0, 1.0], device=DEV)
    B.adamw_step(buf, [g], hyper=torch.tensor([1e-3, 0.1, 0.05, float("nan")], device=DEV), **H)   # nothing
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        B.adamw_step(buf, [g], hyper=hy, **H)
    for t in range(1, 5):
        hy.copy_(torch.tensor([H["lr"] / t, 1 - H["beta1"] ** t, 1 - H["beta2"] ** t, 1.0]))
        gr.replay()
        x = torch.tensor([H["lr"] / t, 1 - H["beta1"] ** t, 1 - H["beta2"] ** t, 1.0], device=DEV)
        B.adamw_step(ref, [h], hyper=x, **H)
        torch.cuda.synchronize()
        assert torch.equal(p, q) and torch.equal(buf.m[0], ref.m[0]) and torch.equal(buf.v[0], ref.v[0])


def test_parameters_that_moved(B):
    """A parameter whose storage was exchanged is stepped where it is now, and refused where it no
    longer fits."""
    p, g, buf = _one(B, "f32", 400)
    old = p.data.clone()
    elsewhere = old.clone()
    first = p.data
    p.data = elsewhere
    B.adamw_step(buf, [g], step=1, **H)
    assert torch.equal(first, old) and not torch.equal(elsewhere, old)
    for bad in (elsewhere[:300], elsewhere.bfloat16(), elsewhere.cpu(), torch.zeros(800, device=DEV)[::2]):
        p.data = bad
        with pytest.raises(B.MoEError) as ei:
            B.adamw_step(buf, [g], step=2, **H)
        assert ei.value.status == 2
    p.data = buf.m[0]
    with pytest.raises(B.MoEError):     # over the step's own moments
        B.adamw_step(buf, [g], step=2, **H)
    p.data = elsewhere
    for bad in (g[:300], g.bfloat16().double(), g.cpu(), torch.zeros(800, device=DEV)[::2]):
        with pytest.raises(B.MoEError) as ei:
            B.adamw_step(buf, [bad], step=2, **H)
        assert ei.value.status == 2


def test_a_tensor_longer_than_a_launch(B):
    """2^33 elements fill a launch; what is behind goes on in another, with the next tensor.
    Codes, scales and offsets past 32 bits, looked at round the ends."""
    n, more = (1 << 33) + 1000, 300
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    print("case adamw 2^33 elements", flush=True)
    at = [0, 4_000_000_000, (1 << 32) - 500, (1 << 33) - 500, n - 700]
    P = [torch.full((s,), 0.5, dtype=torch.bfloat16, device=DEV) for s in (n, more)]
    G = [torch.zeros(s, dtype=torch.bfloat16, device=DEV) for s in (n, more)]
    r = torch.randn(700, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    for a in at:
        G[0][a:a + 700] = r
    G[1][:] = r[:more]
    buf = B.AdamWBuffers.allocate(P, state="8bit")
    B.adamw_step(buf, G, step=1, **H)
    old = np.full(700, 0.5)
    w, m, v = oa.step(old, _n(r), 0 * old, 0 * old, t=1, **H)
    for a in at:
        _check_w(_n(P[0][a:a + 700]), w, old, torch.bfloat16)
    _check_w(_n(P[1]), w[:more], old[:more], torch.bfloat16)
    # without a gradient: the decay alone, moments of zero
    rest = P[0][100_000]
    assert abs(float(rest) - 0.5 * (1 - H["lr"] * H["weight_decay"])) <= 2.0 ** -8 * 0.5
    for a, b in zip(at, at[1:]):
        assert (P[0][a + 700:b] == rest).all() and not buf.m[0][a + 700:b].any()
    for a in at:   # a block's 128 elements share a scale; one wholly inside
        i = -(-a // 128) * 128
        k = slice(i - a, i - a + 128)
        _near_code(buf.m[0][i:i + 128].cpu().numpy(), buf.m_scale[0][i // 128:i // 128 + 1].cpu().numpy(), m[k], False)
        _near_code(buf.v[0][i:i + 128].cpu().numpy(), buf.v_scale[0][i // 128:i // 128 + 1].cpu().numpy(),
                   np.sqrt(v[k]), True)
