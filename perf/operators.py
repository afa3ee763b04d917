"""Cases of the operators a router and its experts train with.

Four operators, each beside the layer's own steps:

* ``balance``      the load-balance loss, the router z-loss and the per-expert counts of a
                   routed batch, per sequence (next to ``moe_route``);
* ``balance_bwd``  their gradient to the logits, in one pass with the routing weights'
                   gradient (next to ``moe_route_bwd``);
* ``ortho``        Newton-Schulz orthogonalisation of a stack of expert gradients (next to
                   the weight gradients of ``moe_bwd``);
* ``muon``         the optimizer step around it: momentum, orthogonalisation and the update
                   of the bf16 expert weights.

``own`` false: the plain form, elementary torch operations. ``own`` true: the library.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
NS = (3.4445, -4.7750, 2.0315)   # the quintic's coefficients
EPS = 1e-7

# S: sequences; tail: tokens behind the last one; drop: share of masked tokens;
# cold: experts switched off by a logit of -inf
_B = dict(S=1, tail=0, drop=0.0, cold=0)


def listed():
    return [
        # one small batch of the tiny layer's router: latency alone
        dict(_B, name="balance_tiny", op="balance", T=64, E=8, k=2),
        # the 16,384-token batch of the 30B-shaped layer, one sequence
        dict(_B, name="balance_30b", op="balance", T=16384, E=128, k=8),
        # a long batch of packed, partly padded sequences over many experts
        dict(_B, name="balance_packed", op="balance", T=131072, E=256, k=8, S=48, tail=500, drop=0.1),
        # the 30B-shaped layer's router backward, renormalised weights
        dict(_B, name="balance_bwd_30b", op="balance_bwd", T=16384, E=128, k=8, renorm=True),
        # an odd batch: rows of 60 logits, nine sequences, two experts off
        dict(_B, name="balance_bwd_odd", op="balance_bwd", T=10007, E=60, k=4, renorm=False, S=9, tail=7, drop=0.2,
             cold=2),
        # the long packed batch again
        dict(_B, name="balance_bwd_packed", op="balance_bwd", T=131072, E=256, k=8, renorm=True, S=48, tail=500,
             drop=0.1),
        # the tiny layer's gate/up gradients: latency alone
        dict(name="ortho_tiny", op="ortho", E=8, R=256, C=256, dtype="bf16"),
        # odd matrices from an fp32 gradient accumulation
        dict(name="ortho_odd_f32", op="ortho", E=6, R=1000, C=777, dtype="f32"),
        # the 30B-shaped layer's down-projection gradients (more rows than columns)
        dict(name="ortho_w2_30b", op="ortho", E=128, R=2048, C=768, dtype="bf16"),
        # the 235B-shaped layer's gate and up gradients, each a matrix of its own
        dict(name="ortho_w13_235b", op="ortho", E=256, R=1536, C=4096, dtype="bf16"),
        # one EP=8 rank's gate/up weights, stacked [gate; up]
        dict(name="muon_w13_ep8", op="muon", E=16, R=1536, C=2048, dtype="bf16", nesterov=False),
        # all gate and up weights of the 30B-shaped layer, each a matrix of its own
        dict(name="muon_w13_30b", op="muon", E=256, R=768, C=2048, dtype="bf16", nesterov=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance_bwd", "ortho", "muon"])
    if op.startswith("balance"):
        while True:
            T, E = _log(rng, 1, 131072), _log(rng, 2, 1024)
            if T * E <= 131072 * 256:
                break
        S = 1 if rng.random() < 0.4 else rng.randint(1, max(1, min(64, T // 2)))
        c = dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 12)), S=S, tail=rng.choice([0, min(T // 3, rng.randint(0, 99))]),
                 drop=rng.choice([0.0, 0.05, 0.3]), cold=rng.choice([0, 0, min(3, E // 4)]))
        c["k"] = min(c["k"], E - c["cold"])
        if op == "balance_bwd":
            c["renorm"] = rng.random() < 0.5
        return c
    while True:
        E, R, C = _log(rng, 1, 64), _log(rng, 4, 4096), _log(rng, 4, 4096)
        if _ns_flops(E, R, C) <= 0.25 * _ns_flops(256, 1536, 4096):
            break
    c = dict(op=op, E=E, R=R, C=C, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "muon":
        c["nesterov"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _router_inputs(c, seed):
    """Logits with Zipf-like popularity, the routing they give, ragged sequence
    bounds, a padding mask, and (backward) the gradients that come in."""
    g = _gen(seed)
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    z = torch.randn((T, E), generator=g, device=DEV)
    rank = torch.randperm(E, generator=g, device=DEV)
    z = z - 0.6 * torch.log1p(rank.float())
    if c["cold"]:
        z[:, rank >= E - c["cold"]] = -math.inf
    v, idx = torch.topk(z, k, dim=1)
    st = {"logits": z.contiguous(), "idx": idx.to(torch.int32).contiguous()}
    n = T - c["tail"]
    cut = torch.sort(torch.randint(0, n + 1, (S - 1,), generator=g, device=DEV)).values
    ends = torch.tensor([0, n], device=DEV)
    st["offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)
    st["mask"] = (torch.rand((T,), generator=g, device=DEV) >= c["drop"]).to(torch.uint8)
    if c["op"] == "balance_bwd":
        renorm = c["renorm"]
        st["w"] = torch.softmax(v, 1) if renorm else torch.exp(v - torch.logsumexp(z, 1, keepdim=True))
        st["w"] = st["w"].contiguous()
        st["dw"] = torch.randn((T, k), generator=g, device=DEV) * 1e-3
        st["dloss"] = torch.tensor([1e-2, 1e-3], device=DEV)
        st["seq_counts"], st["seq_scale"] = _sequence_counts(st, E, k)
    return st


def _sequence_counts(st, E, k):
    """What the forward leaves for the backward: each sequence's counts and its
    factor E / (live sequences * k * live tokens^2); last, 1 / all live tokens."""
    off, S = st["offsets"].long(), st["offsets"].numel() - 1
    T = st["mask"].numel()
    seq = torch.searchsorted(off, torch.arange(T, device=DEV), right=True) - 1
    live = (st["mask"] != 0) & (seq < S)
    pair = (seq[:, None] * E + st["idx"].long())[live].reshape(-1)
    counts = torch.bincount(pair, minlength=S * E)[:S * E].view(S, E)
    n = torch.bincount(seq[live], minlength=S)[:S].double()
    factor = torch.where(n > 0, E / ((n > 0).sum() * k * n * n), torch.zeros_like(n))
    total = n.sum()
    last = torch.where(total > 0, 1.0 / total, torch.zeros_like(total))
    return counts.to(torch.int32).contiguous(), torch.cat([factor, last[None]]).float().contiguous()


def _gradients(c, seed):
    """Expert gradients as a backward leaves them: outer products summed over each
    expert's tokens (some experts saw few, one saw none), channels of uneven
    scale, a magnitude of its own for each expert."""
    g = _gen(seed)
    E, R, C = c["E"], c["R"], c["C"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    r = min(1024, 2 * min(R, C))
    rows = (r * torch.rand((E,), generator=g, device=DEV) ** 0.5).long() + 1
    if E >= 4:
        rows[1] = 0
    out = torch.empty((E, R, C), dtype=dt, device=DEV)
    ch = torch.exp(0.5 * torch.randn((C,), generator=g, device=DEV))
    step = max(1, (1 << 28) // (r * (R + C)))
    for e in range(0, E, step):
        h = min(E, e + step)
        left = torch.randn((h - e, R, r), generator=g, device=DEV)
        right = torch.randn((h - e, r, C), generator=g, device=DEV) * ch
        right *= (torch.arange(r, device=DEV)[None, :] < rows[e:h, None])[:, :, None]
        size = 1e-4 * 10.0 ** torch.randn((h - e, 1, 1), generator=g, device=DEV)
        out[e:h] = torch.bmm(left, right).mul_(size / math.sqrt(r)).to(dt)
    return out, g


def prepare(case, seed):
    c = case
    if c["op"].startswith("balance"):
        st = _router_inputs(c, seed)
    else:
        grad, g = _gradients(c, seed)
        st = {"grad": grad}
        if c["op"] == "muon":
            W = torch.empty((c["E"], c["R"], c["C"]), dtype=torch.bfloat16, device=DEV)
            m = torch.empty((c["E"], c["R"], c["C"]), dtype=torch.float32, device=DEV)
            for e in range(c["E"]):
                W[e] = 0.02 * torch.randn((c["R"], c["C"]), generator=g, device=DEV)
                m[e] = torch.randn((c["R"], c["C"]), generator=g, device=DEV) * grad[e].float().abs().mean()
            st.update(W=W, momentum=m, lr=2e-3, beta=0.95, decay=0.1, scale=0.2 * math.sqrt(max(c["R"], c["C"])))
    st["case"] = dict(c)
    if own:
        from grouped_gemm_02_amd import binding as B
        if c["op"].startswith("balance"):
            st["shape"] = B.make_shape(c["T"], 256, 128, c["E"], c["k"])
            st["buf"] = B.BalanceBuffers.allocate(st["shape"], c["S"])
        else:
            st["shape"] = B.make_ortho_shape(c["E"], c["R"], c["C"], grad=c["dtype"], coeffs=NS, eps=EPS)
            st["buf"] = B.OrthoBuffers.allocate(st["shape"])
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return {"balance": _balance, "balance_bwd": _balance_bwd, "ortho": _ortho, "muon": _muon}[state["case"]["op"]](state)


def _balance(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        b = B.balance(st["buf"], st["logits"], st["idx"], st["offsets"], st["mask"])
        return {"loss": b.loss, "counts": b.counts, "seq_counts": b.seq_counts, "seq_probs": b.seq_probs}
    E, k, S, z = c["E"], c["k"], c["S"], st["logits"]
    off = st["offsets"].long()
    t = torch.arange(z.shape[0], device=DEV)
    live = st["mask"] != 0
    # member[s, t]: whether token t counts in sequence s; the sums of a sequence are
    # products with it over blocks of 256 tokens, joined in 64 bits: the batch is long
    member = (t >= off[:-1, None]) & (t < off[1:, None]) & live
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    s = e.sum(1, keepdim=True)
    lse = (top + torch.log(s))[:, 0]
    hits = torch.zeros_like(z).scatter_add_(1, st["idx"].long(), torch.ones_like(z[:, :k]))
    pad = -z.shape[0] % 256
    blocks = torch.nn.functional.pad(member.float(), (0, pad)).view(S, -1, 256).transpose(0, 1).contiguous()
    rows = torch.nn.functional.pad(torch.cat([e / s, hits], 1), (0, 0, 0, pad)).view(-1, 256, 2 * E)
    sums = torch.bmm(blocks, rows).sum(0, dtype=torch.float64)
    P, counts = sums[:, :E], sums[:, E:].int()
    n = member.sum(1).double()
    zsum = torch.where(member.any(0), lse, torch.zeros_like(lse)).square().sum(dtype=torch.float64)
    some = n > 0
    per = (counts.double() * P).sum(1) * E / (k * n * n)
    balance = torch.where(some, per, torch.zeros_like(per)).sum() / some.sum().clamp(min=1)
    loss = torch.stack([balance, zsum / n.sum().clamp(min=1)]).float()
    return {"loss": loss, "counts": counts.sum(0).int(), "seq_counts": counts,
            "seq_probs": (P / n.clamp(min=1)[:, None]).float()}


def _balance_bwd(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        return B.balance_bwd(st["buf"], st["logits"], st["idx"], st["w"], st["dw"], c["renorm"], st["dloss"],
                             st["offsets"], st["mask"], st["seq_counts"], st["seq_scale"])
    S, z, w, dw = c["S"], st["logits"], st["w"], st["dw"]
    off = st["offsets"].long()
    seq = torch.searchsorted(off, torch.arange(z.shape[0], device=DEV), right=True) - 1
    live = ((st["mask"] != 0) & (seq < S))[:, None]
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    s = e.sum(1, keepdim=True)
    p = e / s
    lse = top + torch.log(s)
    coef = st["seq_counts"].float() * st["seq_scale"][:S, None] * st["dloss"][0]
    G = torch.where(live, coef[seq.clamp(max=S - 1)], torch.zeros_like(p))
    idx = st["idx"].long()
    if not c["renorm"]:
        G = G.scatter_add(1, idx, dw)
    d = p * (G - (p * G).sum(1, keepdim=True))
    d = d + torch.where(live, 2 * st["dloss"][1] * st["seq_scale"][S] * lse, torch.zeros_like(lse)) * p
    if c["renorm"]:
        d = d.scatter_add(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)))
    return d


def _newton_schulz(X):
    """Five steps X <- a X + (b A + c A^2) X with A = X X^T, on the smaller side, in 32 bits."""
    a, b, c = NS
    wide = X.shape[1] <= X.shape[2]
    if not wide:
        X = X.transpose(1, 2).contiguous()
    norm = X.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt()
    X = X / (norm + EPS).float()
    for _ in range(5):
        A = torch.bmm(X, X.transpose(1, 2))
        Bm = torch.baddbmm(A, A, A, beta=b, alpha=c)
        X = torch.baddbmm(X, Bm, X, beta=a)
    return X if wide else X.transpose(1, 2)


def _ortho(st):
    if own:
        from grouped_gemm_02_amd import binding as B
        return B.orthogonalize(st["buf"], st["grad"])
    return _newton_schulz(st["grad"].float()).to(torch.bfloat16).contiguous()


def _muon(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        B.muon_step(st["buf"], st["grad"], st["momentum"], st["W"], lr=st["lr"], momentum_coef=st["beta"],
                    weight_decay=st["decay"], scale=st["scale"], nesterov=c["nesterov"])
        return {"W": st["W"], "momentum": st["momentum"]}
    g, m = st["grad"].float(), st["momentum"]
    m.mul_(st["beta"]).add_(g)
    U = _newton_schulz(g + st["beta"] * m if c["nesterov"] else m)
    W = st["W"].float().mul_(1 - st["lr"] * st["decay"]).sub_(U, alpha=st["lr"] * st["scale"])
    st["W"].copy_(W)
    return {"W": st["W"], "momentum": m}


# ---------------------------------------------------------------- work and exact values

def _ns_flops(E, R, C):
    m, n = min(R, C), max(R, C)
    # A and A^2 are symmetric: one triangle of each
    return E * 5.0 * (m * (m + 1) * n + m * m * (m + 1) + 2.0 * m * m * n)


def work(case):
    c = case
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        return {"bytes": T * (4 * E + 4 * k + 1) + 4 * (S + 1) + 4 * E + 8 * S * E + 8, "flops": 6.0 * T * E}
    if c["op"] == "balance_bwd":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        return {"bytes": T * (8 * E + 12 * k + 1) + 8 * (S + 1) + 4 * S * E + 8, "flops": 9.0 * T * E}
    n = c["E"] * c["R"] * c["C"]
    gb = 2 if c["dtype"] == "bf16" else 4
    extra = 0 if c["op"] == "ortho" else 8 + 2   # momentum read and written, weights read
    return {"bytes": n * (gb + 2 + extra), "flops": _ns_flops(c["E"], c["R"], c["C"])}


def _exact_ns(G, size):
    """The same polynomial in 64 bits by another route: with H = X X^T of the
    normalised input, every iterate is Q X for a polynomial Q of H, so Q is
    built up on the small side alone and applied once."""
    a, b, c = NS
    out = torch.empty(G.shape, dtype=torch.float64, device=DEV)
    for e0 in range(0, G.shape[0], size):
        X = G[e0:e0 + size].double()
        tall = X.shape[1] > X.shape[2]
        X = X.transpose(1, 2).contiguous() if tall else X
        X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + EPS)
        H = torch.bmm(X, X.transpose(1, 2).contiguous())
        eye = torch.eye(H.shape[1], dtype=torch.float64, device=DEV)
        Q = eye.expand_as(H).contiguous()
        for _ in range(5):
            P = a * eye + b * H + c * torch.bmm(H, H)
            Q = torch.bmm(P, Q)
            H = torch.bmm(torch.bmm(P, H), P)
        Y = torch.bmm(Q, X)
        out[e0:e0 + size] = Y.transpose(1, 2) if tall else Y
    return out


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "balance":
        z, idx, off = st["logits"].double(), st["idx"].long(), st["offsets"].tolist()
        probs = torch.zeros((c["S"], c["E"]), dtype=torch.float64, device=DEV)
        total, zsum, alive, used = 0.0, 0.0, 0, 0
        for s in range(c["S"]):
            live = st["mask"][off[s]:off[s + 1]] != 0
            zs, n = z[off[s]:off[s + 1]][live], int(live.sum())
            if n == 0:
                continue
            logp = torch.log_softmax(zs, 1)
            share = torch.bincount(idx[off[s]:off[s + 1]][live].reshape(-1), minlength=c["E"]).double() / (c["k"] * n)
            probs[s] = logp.exp().mean(0)
            total = total + c["E"] * (share * probs[s]).sum()
            zsum = zsum + torch.logsumexp(zs, 1).square().sum()
            alive, used = alive + n, used + 1
        loss = torch.zeros(2, dtype=torch.float64, device=DEV)
        if used:
            loss[0], loss[1] = total / used, zsum / alive
        return {"loss": loss, "counts": None, "seq_counts": None, "seq_probs": probs}
    if c["op"] == "balance_bwd":
        z, idx, off = st["logits"].double(), st["idx"].long(), st["offsets"].tolist()
        p = torch.softmax(z, 1)
        dw, w, gl = st["dw"].double(), st["w"].double(), st["dloss"].double()
        d = torch.zeros_like(p)
        if c["renorm"]:
            d.scatter_(1, idx, w * dw - w * (w * dw).sum(1, keepdim=True))
        else:
            ps = torch.gather(p, 1, idx)
            d.scatter_(1, idx, ps * dw)
            d -= p * (ps * dw).sum(1, keepdim=True)
        scale = st["seq_scale"].double()
        for s in range(c["S"]):
            rows = torch.arange(off[s], off[s + 1], device=DEV)
            rows = rows[st["mask"][rows] != 0]
            if rows.numel() == 0:
                continue
            ps = p[rows]
            v = gl[0] * scale[s] * st["seq_counts"][s].double()
            d[rows] += ps * (v - (ps @ v)[:, None])
            d[rows] += 2 * gl[1] * scale[-1] * torch.logsumexp(z[rows], 1, keepdim=True) * ps
        return d
    m, n = min(c["R"], c["C"]), max(c["R"], c["C"])
    if c["E"] * (10.0 * 2 * m ** 3 * 2 + 4.0 * m * m * n) > 4e14:
        return None
    size = max(1, (1 << 31) // (8 * (8 * m * m + 4 * m * n)))
    if c["op"] == "ortho":
        return _exact_ns(st["grad"], size)
    mom = st["momentum"].double() * st["beta"] + st["grad"].double()
    u = st["grad"].double() + st["beta"] * mom if c["nesterov"] else mom
    U = _exact_ns(u, size)
    W = st["W"].double() * (1 - st["lr"] * st["decay"]) - st["lr"] * st["scale"] * U
    return {"W": W, "momentum": mom}
