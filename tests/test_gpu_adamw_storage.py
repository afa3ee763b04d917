"""The tensors of an AdamW step where their storage, type or strides change between steps."""
import pytest
import torch

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


def _rand(*size, seed=0):
    return torch.randn(size, generator=torch.Generator().manual_seed(seed)).to(DEV)


def test_another_view_of_a_parameters_memory_is_refused(B):
    """The same address and as many elements, but other strides or another type: a step over the
    memory's order would pair elements with others' gradients."""
    for dtype, other in ((torch.float32, torch.int32), (torch.bfloat16, torch.float16)):
        p = _rand(24, 40).to(dtype)
        q = _rand(100, seed=1).to(dtype)
        buf = B.AdamWBuffers.allocate([q, p])
        whole, keep = p.data, p.clone()
        keep_q = q.clone()
        for bad in (whole.t(), whole.view(other)):
            p.data = bad
            assert p.data_ptr() == whole.data_ptr() and p.numel() == whole.numel()
            with pytest.raises(B.MoEError) as ei:
                B.adamw_step(buf, [_rand(100), _rand(*p.shape)], step=1, **H)
            assert ei.value.status == 2
            assert torch.equal(whole, keep) and torch.equal(q, keep_q)
        p.data = whole
        B.adamw_step(buf, [_rand(100), _rand(24, 40)], step=1, **H)
        assert not torch.equal(p, keep)


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_moments_and_masters_that_moved(B, state):
    """What a loaded checkpoint exchanges is stepped where it is now, and what was there is left
    alone; what no longer fits is refused."""
    print(f"case moved moments {state}", flush=True)
    n = 700
    mk = lambda: B.AdamWBuffers.allocate([_rand(n).bfloat16(), _rand(60, seed=2).bfloat16()], state=state, master=True)  # noqa: E731
    buf, ref = mk(), mk()
    names = ["m", "v", "master"] + (["m_scale", "v_scale"] if state == "8bit" else [])
    G = [_rand(n, seed=3), _rand(60, seed=4)]
    for b in (buf, ref):
        B.adamw_step(b, G, step=1, **H)
    first = [(getattr(buf, name)[0].data, getattr(ref, name)[0].clone()) for name in names]
    for name in names:
        t = getattr(buf, name)[0]
        t.data = t.data.clone()
    for b in (buf, ref):
        B.adamw_step(b, G, step=2, **H)
    for old, was in first:
        assert torch.equal(old, was)
    for name in ["params"] + names:
        for a, b in zip(getattr(buf, name), getattr(ref, name)):
            assert torch.equal(a, b), name
    assert not torch.equal(buf.m[0], first[0][0])
    for name in names:
        t = getattr(buf, name)[0]
        good = t.data
        other = torch.float16 if t.dtype == torch.float32 else torch.float32
        for bad in (good[:-1].clone(), good.to(other), good.cpu(), torch.zeros(2 * len(good), dtype=good.dtype, device=DEV)[::2]):
            t.data = bad
            with pytest.raises(B.MoEError) as ei:
                B.adamw_step(buf, G, step=3, **H)
            assert ei.value.status == 2
        t.data = good
    v = buf.v[0].data
    buf.v[0].data = buf.m[0].data   # one over the other
    with pytest.raises(B.MoEError):
        B.adamw_step(buf, G, step=3, **H)
    buf.v[0].data = v
    for b in (buf, ref):
        B.adamw_step(b, G, step=3, **H)
    for name in ["params"] + names:
        for a, b in zip(getattr(buf, name), getattr(ref, name)):
            assert torch.equal(a, b), name


def test_moments_at_an_address_keep_their_memory(B):
    """Memory that a moment left is not given away before the step has looked again: a shorter
    tensor cannot stand at the same address unseen."""
    n = 1 << 20
    p = _rand(n)
    buf = B.AdamWBuffers.allocate([p])
    B.adamw_step(buf, [_rand(n)], step=1, **H)
    at = buf.m[0].data_ptr()
    buf.m[0].data = torch.empty(0, device=DEV)
    short = torch.zeros(n - 1000, device=DEV)
    assert short.data_ptr() != at
    buf.m[0].data = short
    with pytest.raises(B.MoEError):
        B.adamw_step(buf, [_rand(n)], step=2, **H)
    assert not short.any()


@pytest.mark.parametrize("state", ["f32", "8bit"])
def test_gradients_over_what_a_step_writes_are_refused(B, state):
    """A gradient that shares an element with a parameter, a moment, a scale or a master, from
    either side; gradients that touch them only, or share among themselves, are served."""
    print(f"case gradients over buffers {state}", flush=True)
    n = 384
    dt = torch.float32 if state == "f32" else torch.uint8
    w = 4 if state == "f32" else 1
    pool = torch.zeros(64 * n, dtype=torch.uint8, device=DEV)   # one allocation, cut by hand
    at = 0

    def take(count, dtype):
        nonlocal at
        size = count * (torch.finfo(dtype).bits // 8 if dtype.is_floating_point else 1)
        t = pool[at:at + size].view(dtype)
        at += size
        return t
    g0 = take(n, torch.float32)
    p, m, g1, v, master = (take(n, d) for d in (torch.bfloat16, dt, torch.float32, dt, torch.float32))
    ms, vs = (take(4, torch.uint8)[:3] for _ in range(2))
    g2 = take(n, torch.float32)
    buf = B.AdamWBuffers([p], [m], [v], None if state == "f32" else [ms], None if state == "f32" else [vs], [master])
    whole = pool.clone()
    begin = pool.data_ptr()
    for name, t in (("p", p), ("m", m), ("v", v), ("master", master)) + ((("ms", ms), ("vs", vs)) if state == "8bit" else ()):
        first, last = t.data_ptr() - begin, t.data_ptr() - begin + t.numel() * t.element_size()
        for byte in (first, first // 4 * 4 - 4 * n + 4, (last - 1) // 4 * 4):
            if byte < 0:
                continue
            bad = pool[byte:byte + 4 * n].view(torch.float32)
            with pytest.raises(B.MoEError) as ei:
                B.adamw_step(buf, [bad], step=1, **H)
            assert ei.value.status == 2, (name, byte)
    assert torch.equal(pool, whole)
    for g in (g0, g1, g2, g0):   # right before, between and behind them
        g.fill_(1.0)
        B.adamw_step(buf, [g], step=1, **H)
    # the same place in turn with moved moments: looked over again
    g = _rand(n)
    B.adamw_step(buf, [g], step=2, **H)
    keep = g.clone()
    if state == "f32":
        buf.m[0].data = g
        with pytest.raises(B.MoEError):
            B.adamw_step(buf, [g], step=2, **H)
        assert torch.equal(g, keep)
    two = B.AdamWBuffers.allocate([_rand(n), _rand(n)])
    B.adamw_step(two, [g, g], step=1, **H)   # read alone
    B.adamw_step(two, [None, g], step=1, **H)
    assert torch.equal(g, keep)


def test_steps_without_torchs_own_comparisons(B, monkeypatch):
    """Where this torch lacks them the tensors are looked at one by one, with the same results and
    refusals."""
    P, G = [_rand(300), _rand(5, 7, seed=1)], [_rand(300, seed=2), _rand(5, 7, seed=3)]
    ref = B.AdamWBuffers.allocate([p.clone() for p in P])
    B.adamw_step(ref, G, step=1, **H)
    monkeypatch.setattr(B, "_are_at", lambda ts, at, _: [t.data_ptr() for t in ts] == at)
    monkeypatch.setattr(B._Like, "__call__", lambda self, ts: False)
    buf = B.AdamWBuffers.allocate(P)
    B.adamw_step(buf, G, step=1, **H)
    for a, b in zip(buf.params + buf.m + buf.v, ref.params + ref.m + ref.v):
        assert torch.equal(a, b)
    for bad in ([G[0], G[1].t()], [G[0], G[1].bfloat16()], [G[0][:-1], G[1]], [G[0], G[1].cpu()], [buf.m[0], G[1]]):
        with pytest.raises(B.MoEError) as ei:
            B.adamw_step(buf, bad, step=2, **H)
        assert ei.value.status == 2
    B.adamw_step(buf, [None, G[1]], step=2, **H)
    assert torch.equal(buf.params[0], ref.params[0]) and not torch.equal(buf.params[1], ref.params[1])
