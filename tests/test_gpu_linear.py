"""GPU parity of moe_linear and moe_linear_bwd against the float64 oracle, element by
element. With a = |X| |W|^T + |bias| the fp32 sums of K products are off by at most
(K + 2) 2^-24 a in any order (products of bf16 numbers are exact in fp32). The activations
have slopes of at most 1.13 and are computed to 2^-20 of their value; SwiGLU's error is
1.1 |u| dg + |silu(g)| du. One rounding: 2^-8 of the value for bf16, 2^-24 for fp32.
Backward: dP is computed to 2^-19 of the terms it is made of, then rounded to bf16 (2^-8),
which the products carry on."""
import numpy as np
import pytest
import torch

from oracle import moe_linear as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from grouped_gemm_02_amd import binding
    binding.lib()
    return binding


HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _n(t):
    return None if t is None else t.double().cpu().numpy()


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g)


def _forward(B, M, N, K, act, out, bias, residual, pre, seed=0, buf=None):
    print(f"case linear M={M} N={N} K={K} {act} {out} bias={bias} residual={residual} pre={pre}", flush=True)
    r = _rand(seed + M + N + K)
    R = 2 * N if act == "swiglu" else N
    X, W = r(M, K).bfloat16().to(DEV), (r(R, K) / K ** 0.5).bfloat16().to(DEV)
    b = r(R).to(DEV) if bias else None
    res = r(M, N).to(TYPES[out]).to(DEV) if residual else None
    shape = B.make_linear_shape(M, N, K, act=act, out=out)
    buf = buf or B.LinearBuffers.allocate(shape)
    # a row behind each result, which has to stay
    Y = torch.full((M + 1, N), 7.0, dtype=TYPES[out], device=DEV)
    P = torch.full((M + 1, R), 7.0, dtype=torch.bfloat16, device=DEV) if pre else None
    assert B.linear(buf, X, W, b, res, Y=Y, pre=P) is Y
    want, wp = ol.linear(_n(X), _n(W), _n(b), _n(res), act)
    a = np.abs(_n(X)) @ np.abs(_n(W)).T + (np.abs(_n(b)) if bias else 0.0)
    e = (K + 2) * 2.0 ** -24 * a
    if act == "swiglu":
        g, u = np.split(wp, 2, axis=1)
        ey = 1.1 * np.abs(u) * e[:, :N] + np.abs(ol.activate(g, "silu")) * e[:, N:] + e[:, :N] * e[:, N:]
    else:
        ey = 1.13 * e
    body = np.abs(want if res is None else want - _n(res))
    tol = ey + 2.0 ** -20 * body + 2.0 ** -24 * np.abs(want) + HALF[out] * (np.abs(want) + ey) + 1e-37
    off = np.abs(_n(Y[:M]) - want)
    assert np.all(off <= tol), float(np.max(off / tol))
    assert (Y[M] == 7).all()
    if pre:
        assert np.all(np.abs(_n(P[:M]) - wp) <= e + 2.0 ** -8 * (np.abs(wp) + e))
        assert (P[M] == 7).all()
    return Y[:M]


# (M, N, K): single tokens, few rows, ragged tiles of every kind, long and short k
SHAPES = [(1, 1, 1), (1, 8, 16), (1, 768, 2048), (1, 777, 1001), (2, 300, 513), (3, 130, 64), (5, 64, 4096), (16, 1000, 777),
          (17, 256, 1024), (31, 33, 31), (33, 65, 129), (47, 2048, 768), (64, 128, 256), (65, 129, 65), (100, 8, 3000),
          (129, 257, 40), (255, 511, 127), (256, 256, 256), (300, 128, 2048), (1003, 777, 101), (1500, 128, 1024),
          (1024, 1030, 520), (2049, 1025, 200), (4100, 40, 72), (20000, 8, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_match_oracle(B, M, N, K):
    _forward(B, M, N, K, "none", "bf16", False, False, False)
    _forward(B, M, N, K, "none", "f32", True, True, True)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (9, 65, 127), (70, 97, 64), (300, 260, 200), (700, 520, 136)])
def test_activations_match_oracle(B, act, M, N, K):
    for out in ("bf16", "f32"):
        for bias, residual, pre in ((False, False, False), (True, False, True), (True, True, True), (False, True, False)):
            _forward(B, M, N, K, act, out, bias, residual, pre)


def _backward(B, M, N, K, act, out, which=(True, True, True), seed=0):
    print(f"case linear_bwd M={M} N={N} K={K} {act} {out} {which}", flush=True)
    r = _rand(seed + 3 * M + N + K)
    R = 2 * N if act == "swiglu" else N
    X, W = r(M, K).bfloat16().to(DEV), (r(R, K) / K ** 0.5).bfloat16().to(DEV)
    dY = r(M, N).to(TYPES[out]).to(DEV)
    P = None if act == "none" else (1.5 * r(M, R)).bfloat16().to(DEV)
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act=act, out=out))
    dX = torch.full((M + 1, K), 7.0, dtype=torch.bfloat16, device=DEV) if which[0] else None
    dW = torch.full((R + 1, K), 7.0, dtype=torch.bfloat16, device=DEV) if which[1] else None
    db = torch.full((R + 1,), 7.0, device=DEV) if which[2] else None
    got = B.linear_bwd(buf, dY, X, W, P, dX=dX, dW=dW, dbias=db, need_dX=which[0], need_dW=which[1])
    assert got[0] is dX and got[1] is dW and got[2] is db
    wX, wW, wb, dP = ol.linear_backward(_n(dY), _n(X), _n(W), _n(P), act)
    # the terms of dP's formula: at most 1.13 + |P| * 0.8 of dY (times |u|, |silu| for SwiGLU)
    size = np.abs(dP)
    if act in ("silu", "gelu"):
        size = size + np.abs(_n(dY)) * (1.0 + np.abs(_n(P)))
    elif act == "swiglu":
        g, u = np.split(_n(P), 2, axis=1)
        d = np.abs(_n(dY))
        size = size + np.concatenate([d * np.abs(u) * (1.0 + np.abs(g)), d * np.abs(g)], axis=1)
    e = 2.0 ** -19 * size
    ebf = e + 2.0 ** -8 * np.abs(dP)
    aP, aX, aW = np.abs(dP) + ebf, np.abs(_n(X)), np.abs(_n(W))
    if which[0]:
        t = ebf @ aW + (R + 2) * 2.0 ** -24 * (aP @ aW)
        assert np.all(np.abs(_n(dX[:M]) - wX) <= t + 2.0 ** -8 * (np.abs(wX) + t) + 1e-37)
        assert (dX[M] == 7).all()
    if which[1]:
        t = ebf.T @ aX + (M + 2) * 2.0 ** -24 * (aP.T @ aX)
        assert np.all(np.abs(_n(dW[:R]) - wW) <= t + 2.0 ** -8 * (np.abs(wW) + t) + 1e-37)
        assert (dW[R] == 7).all()
    if which[2]:
        t = e.sum(0) + (M + 2) * 2.0 ** -24 * np.abs(dP).sum(0)
        assert np.all(np.abs(_n(db[:R]) - wb) <= t + 1e-37)
        assert (db[R] == 7).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradients_match_oracle(B, M, N, K):
    _backward(B, M, N, K, "none", "bf16")
    _backward(B, M, N, K, "gelu", "f32")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(1, 100, 300), (9, 65, 127), (300, 260, 200), (700, 520, 136)])
def test_gradients_of_activations(B, act, M, N, K):
    for out in ("bf16", "f32"):
        for which in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
            _backward(B, M, N, K, act, out, which)


@pytest.mark.parametrize("act", ["silu", "gelu", "swiglu", "relu"])
def test_gradients_against_differences(B, act):
    """Central differences of the oracle's forward, in the direction of each gradient."""
    M, N, K = 20, 24, 16
    r = _rand(11)
    R = 2 * N if act == "swiglu" else N
    X, W, dY = r(M, K).bfloat16(), (0.5 * r(R, K)).bfloat16(), r(M, N).bfloat16()
    b = r(R)
    x, w, d, bb = (t.double().numpy() for t in (X, W, dY, b))
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act=act))
    P = torch.empty((M, R), dtype=torch.bfloat16, device=DEV)
    B.linear(buf, X.to(DEV), W.to(DEV), b.to(DEV), pre=P)
    dX, dW, db = B.linear_bwd(buf, dY.to(DEV), X.to(DEV), W.to(DEV), P, bias=True)
    f = lambda x, w, bb: float((ol.linear(x, w, bb, None, act)[0] * d).sum())  # noqa: E731
    h = 1e-5
    g = _rand(3)
    for got, at in ((dX, 0), (dW, 1), (db, 2)):
        v = g(*got.shape).double().numpy()
        args = [[x, w, bb], [x, w, bb]]
        args[0][at], args[1][at] = args[0][at] + h * v, args[1][at] - h * v
        diff = (f(*args[0]) - f(*args[1])) / (2 * h)
        mine = float((_n(got) * v).sum())
        # P, dP and the result each rounded to bf16 (2^-8), independently over the elements
        assert abs(diff - mine) <= 4 * 2.0 ** -8 * float(np.linalg.norm(_n(got) * v)) * 2 + 1e-3 * abs(diff)


def test_residual_in_place(B):
    """Y over its residual: the routed experts' result, added to where it is."""
    for M, N, K in ((1, 64, 128), (30, 256, 512), (700, 512, 256)):
        r = _rand(M)
        X, W = r(M, K).bfloat16().to(DEV), (r(N, K) / 16).bfloat16().to(DEV)
        y = r(M, N).bfloat16().to(DEV)
        buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K))
        want = B.linear(buf, X, W, None, y.clone())
        assert B.linear(buf, X, W, None, y, Y=y) is y
        assert torch.equal(y, want)


def test_scratch_serves_fewer_rows(B):
    N, K = 300, 1001
    buf = B.LinearBuffers.allocate(B.make_linear_shape(3000, N, K, act="silu"))
    for M in (1, 2, 63, 500, 1023, 2999):
        r = _rand(M)
        X, W = r(M, K).bfloat16().to(DEV), (r(N, K) / 32).bfloat16().to(DEV)
        own = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act="silu"))
        P, Q = (torch.empty((M, N), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        assert torch.equal(B.linear(buf, X, W, pre=P), B.linear(own, X, W, pre=Q))
        dY = r(M, N).bfloat16().to(DEV)
        for a, b in zip(B.linear_bwd(buf, dY, X, W, P, bias=True), B.linear_bwd(own, dY, X, W, Q, bias=True)):
            assert torch.equal(a, b)


def test_rows_do_not_reach_each_other(B):
    """NaN and infinities in some rows of X, in W, in what lies behind the tensors:
    only their own results see them."""
    for M, N, K in ((7, 40, 100), (130, 200, 72), (300, 300, 1001)):
        r = _rand(M)
        x, w = r(M + 1, K), r(N + 1, K) / K ** 0.5
        x[M], w[N] = torch.nan, torch.nan     # behind what the shape says
        X, W = x.bfloat16().to(DEV), w.bfloat16().to(DEV)
        buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act="relu"))
        buf.fwd_ws.fill_(0xFF)
        buf.bwd_ws.fill_(0xFF)
        clean = B.linear(buf, X[:M], W[:N])
        assert torch.isfinite(clean).all()
        dY = r(M, N).bfloat16().to(DEV)
        P = r(M, N).bfloat16().to(DEV)
        g = B.linear_bwd(buf, dY, X[:M], W[:N], P, bias=True)
        assert all(torch.isfinite(t).all() for t in g)
        X[3, K - 1] = torch.inf
        W[5, 0] = torch.nan
        Y = B.linear(buf, X[:M], W[:N])
        rows = torch.arange(M, device=DEV) != 3
        cols = torch.arange(N, device=DEV) != 5
        assert torch.equal(Y[rows][:, cols], clean[rows][:, cols])
        assert torch.isnan(Y[:, 5]).all() and not torch.isfinite(Y[3]).all()


def test_no_rows(B):
    N, K = 40, 24
    buf = B.LinearBuffers.allocate(B.make_linear_shape(0, N, K))
    X, W = torch.empty((0, K), dtype=torch.bfloat16, device=DEV), torch.ones((N, K), dtype=torch.bfloat16, device=DEV)
    assert B.linear(buf, X, W).shape == (0, N)
    dY = torch.empty((0, N), dtype=torch.bfloat16, device=DEV)
    dX, dW, db = B.linear_bwd(buf, dY, X, W, bias=True)
    assert dX.shape == (0, K) and not dW.any() and not db.any()


@pytest.mark.parametrize("M,N,K", [(1, 640, 2048), (60, 512, 1024), (2000, 1024, 512), (600, 640, 4096)])
def test_captured_and_on_other_streams(B, M, N, K):
    """Replays and another stream give the eager results, bit for bit; two graphs on
    scratches of their own."""
    r = _rand(M)
    X, W = r(M, K).bfloat16().to(DEV), (r(N, K) / K ** 0.5).bfloat16().to(DEV)
    dY, P = r(M, N).bfloat16().to(DEV), r(M, N).bfloat16().to(DEV)
    shape = B.make_linear_shape(M, N, K, act="gelu")
    buf = B.LinearBuffers.allocate(shape)
    want = [B.linear(buf, X, W).clone()] + [t.clone() for t in B.linear_bwd(buf, dY, X, W, P, bias=True)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [B.linear(buf, X, W, stream=side)] + list(B.linear_bwd(buf, dY, X, W, P, bias=True, stream=side))
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        own = B.LinearBuffers.allocate(shape)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [B.linear(own, X, W)] + list(B.linear_bwd(own, dY, X, W, P, bias=True))
        graphs.append((g, out, own))
    for _ in range(3):
        for g, out, own in graphs:
            for t in out:
                t.zero_()
            g.replay()
            B.linear(buf, X, W)
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_rows_of_another_shape_are_refused(B):
    """Rows in three dimensions or of another length are no batch of fewer rows."""
    M, N, K = 24, 40, 16
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K))
    W = torch.ones((N, K), dtype=torch.bfloat16, device=DEV)
    mk = lambda *s: torch.ones(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    for X in (mk(2, 12, K), mk(M * K), mk(12, 2 * K), mk(K, M), mk(M + 1, K)):
        with pytest.raises(B.MoEError) as ei:
            B.linear(buf, X, W)
        assert ei.value.status == 2
    for dY in (mk(2, 12, N), mk(M * N), mk(12, 2 * N), mk(M + 1, N)):
        with pytest.raises(B.MoEError) as ei:
            B.linear_bwd(buf, dY, mk(M, K), W)
        assert ei.value.status == 2
    assert B.linear(buf, mk(3, K), W).shape == (3, N)


def test_offsets_past_32_bits(B):
    """Results and operands of more than 2^31 elements: rows at the ends, round the border and
    between them against the oracle, the row behind them left alone."""
    M, L, S = 600_001, 4096, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    print("case linear past 32 bits", flush=True)
    border = (1 << 31) // L
    rows = torch.tensor([0, 1, border // 2, border - 1, border, border + 1, M - 2, M - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    n = lambda *sz: torch.randn(sz, generator=g, device=DEV)  # noqa: E731
    # a long row out, a residual in place
    X, W, b = n(M, S).bfloat16(), (n(L, S) / 8).bfloat16(), n(L)
    Y = torch.empty((M + 1, L), dtype=torch.bfloat16, device=DEV)
    for at in range(0, M + 1, 50_000):
        Y[at:at + 50_000] = n(*Y[at:at + 50_000].shape).bfloat16()
    old, behind = Y[rows].clone(), Y[M].clone()
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, L, S))
    B.linear(buf, X, W, b, Y[:M], Y=Y[:M])
    want, _ = ol.linear(_n(X[rows]), _n(W), _n(b), _n(old))
    e = (S + 4) * 2.0 ** -24 * (np.abs(_n(X[rows])) @ np.abs(_n(W)).T + np.abs(_n(b)) + np.abs(_n(old)))
    assert np.all(np.abs(_n(Y[rows]) - want) <= e + 2.0 ** -8 * (np.abs(want) + e))
    assert torch.equal(Y[M], behind)
    # backwards from such rows: dX from dY of that size, dW and dbias over all of them
    dY = Y[:M]
    dX, dW, db = B.linear_bwd(buf, dY, X, W, bias=True)
    w = _n(dY[rows]) @ _n(W)
    e = (L + 2) * 2.0 ** -24 * (np.abs(_n(dY[rows])) @ np.abs(_n(W)))
    assert np.all(np.abs(_n(dX[rows]) - w) <= e + 2.0 ** -8 * (np.abs(w) + e))
    cols = torch.tensor([0, 1, L // 2, L - 1], device=DEV)
    d = torch.cat([dY[at:at + 50_000, cols].double() for at in range(0, M, 50_000)]).cpu().numpy()
    x = _n(X)
    e = (M + 2) * 2.0 ** -24 * (np.abs(d).T @ np.abs(x))
    w = d.T @ x
    assert np.all(np.abs(_n(dW[cols]) - w) <= e + 2.0 ** -8 * (np.abs(w) + e))
    assert np.all(np.abs(_n(db[cols]) - d.sum(0)) <= (M + 2) * 2.0 ** -24 * np.abs(d).sum(0))
    # and long rows in, of an odd length (they are copied first)
    del Y, dY, dX
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, S, L - 3, act="relu"), training=False)
    X, W = torch.empty((M, L - 3), dtype=torch.bfloat16, device=DEV), (n(S, L - 3) / 64).bfloat16()
    for at in range(0, M, 50_000):
        X[at:at + 50_000] = n(*X[at:at + 50_000].shape).bfloat16()
    Y = B.linear(buf, X, W)
    want, _ = ol.linear(_n(X[rows]), _n(W), act="relu")
    e = (L + 2) * 2.0 ** -24 * (np.abs(_n(X[rows])) @ np.abs(_n(W)).T)
    assert np.all(np.abs(_n(Y[rows]) - want) <= e + 2.0 ** -8 * (np.abs(want) + e))


@pytest.mark.parametrize("M,N,K", [(300, 640, 4096), (1003, 257, 1001), (3000, 96, 203)])   # parts, copies, both
def test_two_graphs_share_a_scratch(B, M, N, K):
    """Two captured passes over one scratch, replayed in turn and between eager calls on it, with
    inputs that change: nothing is left in it that a later call relies on."""
    print(f"case two graphs, one scratch {M} {N} {K}", flush=True)
    buf = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act="silu"))
    own = B.LinearBuffers.allocate(B.make_linear_shape(M, N, K, act="silu"))
    sets = []
    for s, rows in ((1, M), (2, M // 2 + 1)):
        r = _rand(s)
        sets.append([r(rows, K).bfloat16().to(DEV), (r(N, K) / K ** 0.5).bfloat16().to(DEV), r(rows, N).bfloat16().to(DEV),
                     r(rows, N).bfloat16().to(DEV)])
    both = lambda b, X, W, dY, P: [B.linear(b, X, W)] + list(B.linear_bwd(b, dY, X, W, P, bias=True))  # noqa: E731
    both(buf, *sets[0])
    torch.cuda.synchronize()
    graphs = []
    for a in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(buf, *a)
        graphs.append((g, out))
    for _ in range(3):
        for a in sets:
            for t in a:
                t.copy_(t.roll(1, 0))
        for i in (0, 1, 0):
            graphs[i][0].replay()
        both(buf, *sets[1])
        torch.cuda.synchronize()
        for (_, out), a in zip(graphs, sets):
            for x, y in zip(out, both(own, *a)):
                assert torch.equal(x, y)
