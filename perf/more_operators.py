"""Cases of the operators around the layer: the router's product and its choice of
experts, a shared expert's products, and the optimizer of everything that is not
orthogonalised.

* ``gate``        experts by softmax or sigmoid scores, with a bias for balance, groups, top-k
                  and renormalised weights (next to ``moe_route``);
* ``gate_bwd``    its gradient to the logits (next to ``moe_route_bwd``);
* ``linear``      a dense product with bias, activation and residual (the router's logits, a
                  shared expert whose result joins the routed experts');
* ``linear_bwd``  its gradients;
* ``adamw``       an AdamW step over many tensors at once, moments in 32 or in 8 bits (next to
                  ``moe_muon_step``).

``own`` false: the plain form, elementary torch operations. ``own`` true: the library.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # values that share a scale where the moments are held in 8 bits
GELU = (math.sqrt(2.0 / math.pi), 0.044715)

# score: softmax or sigmoid; G: groups, L: groups kept, top: scores that make a group's;
# drop: share of masked tokens; cold: experts switched off by a logit of -inf;
# train: what stands before the activation is kept for the gradient
_G = dict(score="softmax", bias=False, renorm=True, G=1, L=1, top=1, scale=1.0, drop=0.0, cold=0)
_L = dict(act="none", out="bf16", bias=False, residual=False, train=False)


def listed():
    return [
        # one small batch of the tiny layer's router: latency alone
        dict(_G, name="gate_tiny", op="gate", T=64, E=8, k=2),
        # the 16,384-token batch of the 30B-shaped layer, sigmoid scores with a bias for balance
        dict(_G, name="gate_30b_bias", op="gate", T=16384, E=128, k=8, score="sigmoid", bias=True),
        # a long padded batch over many experts in groups, the best four groups of eight
        dict(_G, name="gate_groups", op="gate", T=131072, E=256, k=8, score="sigmoid", bias=True, G=8, L=4, top=2,
             scale=2.5, drop=0.1),
        # the gradient of the 30B-shaped layer's choice
        dict(_G, name="gate_bwd_30b", op="gate_bwd", T=16384, E=128, k=8, score="sigmoid", bias=True),
        # an odd batch, all probabilities in the gradient, two experts off
        dict(_G, name="gate_bwd_odd", op="gate_bwd", T=100007, E=60, k=4, renorm=False, drop=0.2, cold=2),
        # one token of a server through a shared expert's gate and up product
        dict(_L, name="linear_one_token", op="linear", M=1, N=768, K=2048, act="swiglu"),
        # the router's product over the 30B-shaped layer's batch, logits in 32 bits
        dict(_L, name="linear_router", op="linear", M=16384, N=128, K=2048, out="f32"),
        # a shared expert's down product of the 235B-shaped layer, added to the routed experts' result
        dict(_L, name="linear_down", op="linear", M=16384, N=4096, K=1536, residual=True),
        # odd sizes in every place
        dict(_L, name="linear_bwd_odd", op="linear_bwd", M=1003, N=777, K=1001, act="gelu", bias=True),
        # a shared expert's gate and up product of the 30B-shaped layer
        dict(_L, name="linear_bwd_up", op="linear_bwd", M=16384, N=768, K=2048, act="swiglu"),
        # the routers and biases of 48 layers in 32 bits
        dict(name="adamw_routers", op="adamw", tensors=96, numel=12589056, param="f32", grad="f32", state="f32",
             master=False, clip=True),
        # one 30B-shaped layer's expert weights, moments in 8 bits
        dict(name="adamw_experts_8bit", op="adamw", tensors=2, numel=603979776, param="bf16", grad="bf16",
             state="8bit", master=False, clip=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "gate_bwd", "linear", "linear_bwd", "adamw"])
    if op.startswith("gate"):
        while True:
            T, E = _log(rng, 1, 131072), _log(rng, 2, 1024)
            if T * E <= 131072 * 256:
                break
        G = rng.choice([g for g in (1, 1, 2, 4, 5, 8, 16) if E % g == 0 and E // g >= 2] or [1])
        L = rng.randint(1, G)
        k = rng.randint(1, min(12, L * (E // G)))
        cold = rng.choice([0, 0, min(3, E // 4)])
        return dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    renorm=rng.random() < 0.6, G=G, L=L, top=rng.choice([1, 2]) if G > 1 else 1,
                    scale=rng.choice([1.0, 2.5]), drop=rng.choice([0.0, 0.05, 0.3]), cold=cold)
    if op.startswith("linear"):
        while True:
            M, N, K = _log(rng, 1, 16384), _log(rng, 8, 4096), _log(rng, 16, 4096)
            if M * N * K <= 16384 * 4096 * 1536 // 4:
                break
        act = rng.choice(["none", "none", "relu", "silu", "gelu", "swiglu"])
        return dict(op=op, M=M, N=N, K=K, act=act, out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5,
                    residual=op == "linear" and rng.random() < 0.5,
                    train=op == "linear" and act != "none" and rng.random() < 0.5)
    param = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, tensors=_log(rng, 1, 200), numel=_log(rng, 1000, 100000000), param=param,
                grad=rng.choice(["bf16", "f32"]), state=rng.choice(["f32", "8bit"]),
                master=param == "bf16" and rng.random() < 0.5, clip=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gate_inputs(c, seed):
    """Logits with Zipf-like popularity, a bias as balancing leaves it (popular
    experts pushed down), a padding mask; for the gradient a choice of experts and
    what comes back to their weights."""
    g = _gen(seed)
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.randn((T, E), generator=g, device=DEV)
    rank = torch.randperm(E, generator=g, device=DEV)
    z = z - 0.6 * torch.log1p(rank.float())
    if c["cold"]:
        z[:, rank >= E - c["cold"]] = -math.inf
    st = {"logits": z.contiguous(), "bias": None, "mask": None}
    if c["bias"]:
        typical = 0.15 if c["score"] == "sigmoid" else 1.0 / E
        st["bias"] = typical * (0.2 * torch.log1p(rank.float()) + 0.3 * torch.randn((E,), generator=g, device=DEV))
    if c["drop"]:
        st["mask"] = (torch.rand((T,), generator=g, device=DEV) >= c["drop"]).to(torch.uint8)
    if c["op"] == "gate_bwd":
        idx = _choose(c, z, st["bias"], st["mask"])[0]
        st["idx"] = idx.to(torch.int32).contiguous()
        st["dw"] = torch.randn((T, k), generator=g, device=DEV) * 1e-3
    return st


def _linear_inputs(c, seed):
    g = _gen(seed)
    M, N, K = c["M"], c["N"], c["K"]
    rows = 2 * N if c["act"] == "swiglu" else N
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    ch = torch.exp(0.5 * rand(K))   # channels of uneven size, as a norm's gain leaves them
    st = {"X": (rand(M, K) * ch).bfloat16(), "W": (rand(rows, K) / math.sqrt(K)).bfloat16()}
    st["bias"] = 0.3 * rand(rows) if c["bias"] else None
    if c["op"] == "linear":
        st["residual"] = rand(M, N).to(_type(c["out"])) if c["residual"] else None
        st["kept"] = torch.empty((M, rows), dtype=torch.bfloat16, device=DEV) if c["train"] else None
    else:
        st["dY"] = (rand(M, N) * 1e-3).to(_type(c["out"]))
        st["pre"] = None if c["act"] == "none" else rand(M, rows).bfloat16()
    return st


def _sizes(c):
    """Tensors of uneven sizes, the sum near numel."""
    q = [2 ** (5 * i % 7) for i in range(c["tensors"])]
    return [max(1, c["numel"] * v // sum(q)) for v in q]


def _blocks(n):
    return -(-n // BLOCK)


def _adamw_inputs(c, seed):
    """The tensors lie one after the other in flat buffers; in 8 bits each one's
    moments begin a block."""
    g = _gen(seed)
    sizes = _sizes(c)
    n = sum(sizes)
    st = {"sizes": sizes}
    w = torch.randn((n,), generator=g, device=DEV)
    w *= 0.02
    st["param"] = w.to(_type(c["param"]))
    st["master"] = w if c["master"] else None
    if c["param"] == "f32" and not c["master"]:
        st["param"] = w
    st["grad"] = torch.empty((n,), dtype=_type(c["grad"]), device=DEV)
    size = 1e-4 * torch.exp(torch.randn((len(sizes),), generator=g, device=DEV))
    at = 0
    for i, s in enumerate(sizes):
        st["grad"][at:at + s] = torch.randn((s,), generator=g, device=DEV).mul_(size[i])
        at += s
    if c["state"] == "f32":
        st["m"] = 0.3e-4 * torch.randn((n,), generator=g, device=DEV)
        st["v"] = (1e-4 * torch.randn((n,), generator=g, device=DEV)).square_()
    else:
        b = sum(_blocks(s) for s in sizes)
        for name in ("m", "v"):
            x = torch.randn((b * BLOCK,), generator=g, device=DEV).mul_(0.3e-4 if name == "m" else 1e-4)
            at = 0
            for s in sizes:   # behind a tensor's end its last block holds zeros
                x[at + s:at + _blocks(s) * BLOCK] = 0
                at += _blocks(s) * BLOCK
            st[name], st[name + "_scale"] = _to_8bit(x if name == "m" else x.abs_())
    st["clip"] = torch.tensor([0.37], device=DEV) if c["clip"] else None
    st["hyper"] = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1000)
    return st


def prepare(case, seed):
    c = case
    kind = c["op"].split("_")[0]
    st = {"gate": _gate_inputs, "linear": _linear_inputs, "adamw": _adamw_inputs}[kind](c, seed)
    st["case"] = dict(c)
    if own:
        from grouped_gemm_02_amd import binding as B
        if kind == "gate":
            st["shape"] = B.make_shape(c["T"], 256, 128, c["E"], c["k"])
            st["params"] = B.make_gate_params(c["score"], renorm=c["renorm"], groups=c["G"], groups_kept=c["L"],
                                              group_top=c["top"], scale=c["scale"])
        elif kind == "linear":
            st["shape"] = B.make_linear_shape(c["M"], c["N"], c["K"], act=c["act"], out=c["out"])
            st["buf"] = B.LinearBuffers.allocate(st["shape"])
        else:
            cut = lambda t, s: None if t is None else list(torch.split(t, s))  # noqa: E731
            sizes = st["sizes"]
            if c["state"] == "8bit":
                whole = [_blocks(s) * BLOCK for s in sizes]
                at = [sum(whole[:i]) for i in range(len(sizes))]
                codes = lambda t: [t[a:a + s] for a, s in zip(at, sizes)]  # noqa: E731
                scales = lambda t: list(torch.split(t, [_blocks(s) for s in sizes]))  # noqa: E731
                st["buf"] = B.AdamWBuffers(cut(st["param"], sizes), codes(st["m"]), codes(st["v"]), scales(st["m_scale"]),
                                           scales(st["v_scale"]), cut(st["master"], sizes))
            else:
                st["buf"] = B.AdamWBuffers(cut(st["param"], sizes), cut(st["m"], sizes), cut(st["v"], sizes), None, None,
                                           cut(st["master"], sizes))
            st["grads"] = cut(st["grad"], sizes)
    return st


# ---------------------------------------------------------------- one pass

def run(state):
    return {"gate": _gate, "gate_bwd": _gate_bwd, "linear": _linear, "linear_bwd": _linear_bwd,
            "adamw": _adamw}[state["case"]["op"]](state)


def _choose(c, z, bias, mask):
    """Experts (-1: none left) and their scores in 64 bits: values next to each
    other decide whole numbers."""
    T, E, k, G = z.shape[0], c["E"], c["k"], c["G"]
    x = z.double()
    live = x > -math.inf
    if c["score"] == "softmax":
        e = torch.exp(x - x.max(1, keepdim=True).values)
        s = e / e.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    pick = x if bias is None else torch.where(live, s + bias.double(), x)
    if G > 1:
        by = pick if c["top"] == 1 else torch.where(live, s if bias is None else pick, x)
        best = torch.sort(by.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["top"]]
        score = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        score = torch.where(best[:, :, 0] > -math.inf, score, torch.full_like(score, -math.inf))
        order = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :c["L"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, order, True)
        pick = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), pick, torch.full_like(pick, -math.inf))
    best, idx = torch.sort(pick, dim=1, descending=True, stable=True)
    some = best[:, :k] > -math.inf
    if mask is not None:
        some = some & (mask != 0)[:, None]
    return torch.where(some, idx[:, :k], torch.full_like(idx[:, :k], -1)), s


def _gate(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        idx, w = B.gate(st["shape"], st["params"], st["logits"], st["bias"], st["mask"])
        return {"idx": idx, "w": w}
    idx, s = _choose(c, st["logits"], st["bias"], st["mask"])
    w = torch.where(idx >= 0, torch.gather(s, 1, idx.clamp(min=0)), torch.zeros_like(s[:, :1]))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return {"idx": idx.to(torch.int32), "w": (w * c["scale"]).float()}


def _gate_bwd(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        return B.gate_bwd(st["shape"], st["params"], st["logits"], st["idx"], st["dw"])
    z, idx = st["logits"], st["idx"].long()
    some = idx >= 0
    at = idx.clamp(min=0)
    none = torch.zeros_like(st["dw"])
    dw = torch.where(some, st["dw"], none)
    if c["score"] == "softmax" and not c["renorm"]:
        e = torch.exp(z - z.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
        G = torch.zeros_like(z).scatter_add_(1, at, dw)
        return c["scale"] * p * (G - (p * G).sum(1, keepdim=True))
    zs = torch.gather(z, 1, at)
    if c["score"] == "softmax":
        zs = torch.where(some, zs, torch.full_like(zs, -math.inf))
        top = zs.max(1, keepdim=True).values
        e = torch.where(some, torch.exp(zs - top), none)
        slope = torch.ones_like(e)
    else:
        e = torch.where(some, 1.0 / (1.0 + torch.exp(-zs)), none)
        slope = 1.0 / (1.0 + torch.exp(zs))
    if c["renorm"]:
        total = e.sum(1, keepdim=True)
        e = e / torch.where(total > 0, total, torch.ones_like(total))
        dw = dw - (e * dw).sum(1, keepdim=True)
    d = torch.where(some, c["scale"] * e * slope * dw, none)
    return torch.zeros_like(z).scatter_add_(1, at, d)


def _act(c, P):
    if c["act"] == "relu":
        return torch.where(P > 0, P, torch.zeros_like(P))
    if c["act"] == "silu":
        return P / (1.0 + torch.exp(-P))
    if c["act"] == "gelu":
        return P / (1.0 + torch.exp(-2.0 * GELU[0] * (P + GELU[1] * P * P * P)))
    if c["act"] == "swiglu":
        g, u = P[:, :c["N"]], P[:, c["N"]:]
        return g / (1.0 + torch.exp(-g)) * u
    return P


def _act_bwd(c, dY, P):
    """dL/dP of L with dL/d act(P) = dY."""
    if c["act"] == "none":
        return dY
    if c["act"] == "relu":
        return torch.where(P > 0, dY, torch.zeros_like(dY))
    if c["act"] == "gelu":
        s = 1.0 / (1.0 + torch.exp(-2.0 * GELU[0] * (P + GELU[1] * P * P * P)))
        return dY * (s + P * s * (1.0 - s) * 2.0 * GELU[0] * (1.0 + 3.0 * GELU[1] * P * P))
    g = P[:, :c["N"]]
    s = 1.0 / (1.0 + torch.exp(-g))
    slope = s * (1.0 + g * (1.0 - s))
    if c["act"] == "silu":
        return dY * slope
    u = P[:, c["N"]:]
    return torch.cat([dY * u * slope, dY * g * s], 1)


def _linear(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        return {"Y": B.linear(st["buf"], st["X"], st["W"], bias=st["bias"], residual=st["residual"], pre=st["kept"]),
                "pre": st["kept"]}
    P = st["X"].float() @ st["W"].float().t()
    if st["bias"] is not None:
        P += st["bias"]
    Y = _act(c, P)
    if st["residual"] is not None:
        Y = Y + st["residual"].float()
    if c["train"]:
        st["kept"].copy_(P)
    return {"Y": Y.to(_type(c["out"])), "pre": st["kept"]}


def _linear_bwd(st):
    c = st["case"]
    if own:
        from grouped_gemm_02_amd import binding as B
        dX, dW, db = B.linear_bwd(st["buf"], st["dY"], st["X"], st["W"], pre=st["pre"], bias=c["bias"])
        return {"dX": dX, "dW": dW, "db": db}
    dP = _act_bwd(c, st["dY"].float(), None if st["pre"] is None else st["pre"].float())
    db = dP.sum(0, dtype=torch.float64).float() if c["bias"] else None
    return {"dX": (dP @ st["W"].float()).bfloat16(), "dW": (dP.t() @ st["X"].float()).bfloat16(), "db": db}


def _to_8bit(x):
    """E4M3 codes of whole blocks, and a byte e + 127 for each block: the smallest
    power of two 2^e (e from -126 to 126) with 448 2^e no less than the block's
    largest magnitude; e = 0 for a block of zeros."""
    x = x.view(-1, BLOCK)
    f, e = torch.frexp(x.abs().amax(1))
    e = torch.where(f > 0, (e - 9 + (f > 0.875).int()).clamp(-126, 126), torch.zeros_like(e))
    codes = (x * _power(127 - e)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(-1), (e + 127).to(torch.uint8)


def _power(byte):
    """2^(byte - 127), from its bits."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _from_8bit(codes, scale):
    x = codes.view(torch.float8_e4m3fn).float().view(-1, BLOCK)
    return (x * _power(scale)[:, None]).view(-1)


def _spread(x, sizes):
    """A flat buffer of tensors, each one begun at a block and filled up with zeros."""
    out = torch.zeros((sum(_blocks(s) for s in sizes), BLOCK), dtype=x.dtype, device=DEV).view(-1)
    a = b = 0
    for s in sizes:
        out[b:b + s] = x[a:a + s]
        a, b = a + s, b + _blocks(s) * BLOCK
    return out


def _gather(x, sizes):
    out, b = [], 0
    for s in sizes:
        out.append(x[b:b + s])
        b += _blocks(s) * BLOCK
    return torch.cat(out)


def _answer(st):
    """The state after the step. Moments in 8 bits are the numbers of their codes,
    and each block's power of two."""
    out = {"param": st["param"], "master": st["master"]}
    for name in ("m", "v"):
        if st["case"]["state"] == "f32":
            out[name] = st[name]
        else:
            out[name] = st[name].view(torch.float8_e4m3fn)
            out[name + "_scale"] = st[name + "_scale"].view(torch.float8_e8m0fnu)
    return out


def _adamw(st):
    c, h, sizes = st["case"], st["hyper"], st["sizes"]
    if own:
        from grouped_gemm_02_amd import binding as B
        B.adamw_step(st["buf"], st["grads"], lr=h["lr"], beta1=h["beta1"], beta2=h["beta2"], eps=h["eps"],
                     weight_decay=h["weight_decay"], step=h["step"], grad_scale=st["clip"])
        return _answer(st)
    eight = c["state"] == "8bit"
    g = st["grad"].float()
    if st["clip"] is not None:
        g = g * st["clip"]
    if eight:
        g = _spread(g, sizes)
        m, root = _from_8bit(st["m"], st["m_scale"]), _from_8bit(st["v"], st["v_scale"])
        v = root * root
    else:
        m, v = st["m"], st["v"]
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + g * (1.0 - h["beta2"]) * g
    root = torch.sqrt(v)
    size = h["lr"] / (1.0 - h["beta1"] ** h["step"])
    update = m * size / (root * (1.0 / math.sqrt(1.0 - h["beta2"] ** h["step"])) + h["eps"])
    w = st["param"].float() if st["master"] is None else st["master"]
    w = w * (1.0 - h["lr"] * h["weight_decay"]) - (_gather(update, sizes) if eight else update)
    if st["master"] is not None:
        st["master"].copy_(w)
    st["param"].copy_(w)
    if eight:
        for name, x in (("m", m), ("v", root)):
            codes, scale = _to_8bit(x)
            if name == "v":   # a root that is not zero is not held as zero: steps divide by it
                codes = torch.where((x > 0) & (codes == 0), torch.ones_like(codes), codes)
            st[name].copy_(codes)
            st[name + "_scale"].copy_(scale)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return _answer(st)


# ---------------------------------------------------------------- work and exact values

def work(case):
    c = case
    if c["op"] == "gate":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * (4 * E + 8 * k) + (T if c["drop"] else 0) + (4 * E if c["bias"] else 0),
                "flops": 5.0 * T * E}
    if c["op"] == "gate_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * (4 * E + 8 * k + 4 * (E if dense else k)), "flops": T * (7.0 * E if dense else 12.0 * k)}
    if c["op"].startswith("linear"):
        M, N, K = c["M"], c["N"], c["K"]
        rows = 2 * N if c["act"] == "swiglu" else N
        sz = 2 if c["out"] == "bf16" else 4
        once = 2 * M * K + 2 * rows * K + (4 * rows if c["bias"] else 0)
        if c["op"] == "linear":
            return {"bytes": once + sz * M * N * (2 if c["residual"] else 1) + (2 * M * rows if c["train"] else 0),
                    "flops": 2.0 * M * rows * K}
        return {"bytes": once + 2 * M * K + 2 * rows * K + sz * M * N + (2 * M * rows if c["act"] != "none" else 0),
                "flops": 4.0 * M * rows * K}
    n = sum(_sizes(c))
    size = {"bf16": 2, "f32": 4}
    moments = 16 if c["state"] == "f32" else 4 + 4.0 / BLOCK
    weights = size[c["param"]] + (8 if c["master"] else size[c["param"]])
    return {"bytes": n * (size[c["grad"]] + weights + moments), "flops": 16.0 * n}


def _exact_gate(c, st):
    """One expert at a time, the largest that is left, ties to the lower id."""
    z = st["logits"].double()
    T, E, k, G = z.shape[0], c["E"], c["k"], c["G"]
    lowest = torch.full((), -math.inf, dtype=torch.float64, device=DEV)
    if c["score"] == "softmax":
        s = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    else:
        s = torch.where(z >= 0, 1 / (1 + torch.exp(-z)), torch.exp(z) / (1 + torch.exp(z)))
    off = torch.isinf(z)
    c1 = z if st["bias"] is None else s + st["bias"].double()
    c2 = s if st["bias"] is None else c1
    c1, c2 = torch.where(off, lowest, c1), torch.where(off, lowest, c2)
    ids = torch.arange(E, device=DEV)

    def largest(x, n):
        where = torch.arange(n, device=DEV)
        top = x.max(-1, keepdim=True).values
        return top[..., 0], torch.where(x == top, where, n).min(-1).values

    if G > 1:
        by = (c1 if c["top"] == 1 else c2).view(T, G, E // G)
        a, i = largest(by, E // G)
        score = a
        if c["top"] == 2:
            rest = torch.where(torch.arange(E // G, device=DEV) == i[..., None], lowest, by)
            b = rest.max(-1).values
            score = torch.where(torch.isinf(b), a, a + b)
        kept = torch.zeros((T, G), dtype=torch.bool, device=DEV)
        for _ in range(c["L"]):
            _, g = largest(score, G)
            hit = torch.arange(G, device=DEV) == g[:, None]
            kept |= hit
            score = torch.where(hit, lowest, score)
        c1 = torch.where(kept.repeat_interleave(E // G, dim=1), c1, lowest)
    w = torch.zeros((T, k), dtype=torch.float64, device=DEV)
    for j in range(k):
        v, i = largest(c1, E)
        some = ~torch.isinf(v)
        if st["mask"] is not None:
            some &= st["mask"] != 0
        w[:, j] = torch.where(some, torch.gather(s, 1, i.clamp(max=E - 1)[:, None])[:, 0], torch.zeros_like(v))
        c1 = torch.where(ids == i[:, None], lowest, c1)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    return {"idx": None, "w": w * c["scale"]}


def _exact_gate_bwd(c, st):
    """Through the scores: dL/ds first, then the scores' own derivatives."""
    z, idx, dw = st["logits"].double(), st["idx"].long(), st["dw"].double() * c["scale"]
    hit = torch.zeros_like(z)
    D = torch.zeros_like(z)
    for j in range(c["k"]):
        e = idx[:, j:j + 1]
        some = (e >= 0).double()
        hit.scatter_add_(1, e.clamp(min=0), some)
        D.scatter_add_(1, e.clamp(min=0), dw[:, j:j + 1] * some)
    s = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
    if c["renorm"]:
        total = (s * hit).sum(1, keepdim=True)
        some = (total > 0).double()
        total = total + (1 - some)
        D = some * hit * (D / total - (s * D).sum(1, keepdim=True) / total ** 2)
    if c["score"] == "softmax":
        return s * (D - (s * D).sum(1, keepdim=True))
    return s * torch.sigmoid(-z) * D


def _exact_act(c, P):
    if c["act"] == "relu":
        return P.clamp(min=0)
    if c["act"] == "silu":
        return P * torch.sigmoid(P)
    if c["act"] == "gelu":
        return 0.5 * P * (1 + torch.tanh(GELU[0] * (P + GELU[1] * P ** 3)))
    if c["act"] == "swiglu":
        g, u = P.chunk(2, 1)
        return g * torch.sigmoid(g) * u
    return P


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "gate":
        return _exact_gate(c, st)
    if c["op"] == "gate_bwd":
        return _exact_gate_bwd(c, st)
    if c["op"] == "linear":
        P = torch.mm(st["X"].double(), st["W"].double().t().contiguous())
        if st["bias"] is not None:
            P += st["bias"].double()
        Y = _exact_act(c, P)
        return {"Y": Y if st["residual"] is None else Y + st["residual"].double(), "pre": P if c["train"] else None}
    if c["op"] == "linear_bwd":
        dY = st["dY"].double()
        if st["pre"] is None:
            dP = dY
        else:   # the slope of the activation by its own derivative, column by column of ones
            P = st["pre"].double().requires_grad_(True)
            dP = torch.autograd.grad(_exact_act(c, P), P, dY)[0]
        return {"dX": torch.mm(dP, st["W"].double()), "dW": torch.mm(dP.t().contiguous(), st["X"].double()),
                "db": dP.sum(0) if c["bias"] else None}
    h, n = st["hyper"], st["param"].numel()
    out = {"param": torch.empty((n,), dtype=torch.float64, device=DEV), "master": None}
    if c["state"] == "f32":
        out["m"], out["v"] = torch.empty_like(out["param"]), torch.empty_like(out["param"])
    else:   # codes next to a border go either way: the moments are held to their type
        out.update(m=None, v=None, m_scale=None, v_scale=None)
    clip = 1.0 if st["clip"] is None else float(st["clip"])
    a = b = blk = 0
    for s in st["sizes"]:
        g = st["grad"][a:a + s].double() * clip
        if c["state"] == "f32":
            m, v = st["m"][a:a + s].double(), st["v"][a:a + s].double()
        else:
            q = _blocks(s)
            e = lambda t: torch.exp2(t[blk:blk + q].double() - 127).repeat_interleave(BLOCK)[:s]  # noqa: E731
            num = lambda t: t[b:b + s].view(torch.float8_e4m3fn).double()  # noqa: E731
            m, v = num(st["m"]) * e(st["m_scale"]), (num(st["v"]) * e(st["v_scale"])) ** 2
            b, blk = b + q * BLOCK, blk + q
        m = h["beta1"] * m + (1 - h["beta1"]) * g
        v = h["beta2"] * v + (1 - h["beta2"]) * g ** 2
        w = (st["param"] if st["master"] is None else st["master"])[a:a + s].double()
        mh, vh = m / (1 - h["beta1"] ** h["step"]), v / (1 - h["beta2"] ** h["step"])
        out["param"][a:a + s] = w - h["lr"] * (mh / (vh.sqrt() + h["eps"]) + h["weight_decay"] * w)
        if c["state"] == "f32":
            out["m"][a:a + s], out["v"][a:a + s] = m, v
        a += s
    if c["master"]:
        out["master"] = out["param"]
    return out
