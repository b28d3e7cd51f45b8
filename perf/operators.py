"""The feed-forward half of a decode step around the W8A8 linear layers, as a
list of timed cases: the norms between two blocks with the quantiser behind
them, the router, and the experts of a few tokens.

run(state) computes a case either in its plain form (elementary torch
operations in 32 bits, the router in 64) or, where `own` is true, through the
library's entry points norm_residual_quant, moe_route_topk and
moe_w8a8_block.  exact(case, seed) is the definition in 64 bits.
"""

import math

import torch

own = False

GROUP = 128
HALF = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _w8():
    import w8a8_int8_quantized_amd as w8
    return w8


# ------------------------------------------------------------------- cases
def _moe(name, T, K, I, E, topk, local=1.0):
    return {"name": name, "op": "moe", "T": T, "K": K, "I": I, "E": E, "topk": topk, "local": local}


def _route(name, T, E, topk, score, groups=1, kept=1, dtype="fp32", bias=False, masked=0.0):
    return {"name": name, "op": "route", "T": T, "E": E, "topk": topk, "score": score, "groups": groups, "kept": kept,
            "dtype": dtype, "bias": bias, "masked": masked}


def _norm(name, M, K, out, dtype="bf16", residual=True, post=False, gate="none", scale=1.0):
    return {"name": name, "op": "norm", "M": M, "K": K, "out": out, "dtype": dtype, "residual": residual, "post": post,
            "gate": gate, "scale": scale}


def listed():
    return [
        # one request being answered, a small model: what counts is the latency of the launches
        _moe("moe small 1 token", 1, 1024, 256, 16, 2),
        # one request, the experts of a DeepSeek-V3 layer: eight experts' weights pass once
        _moe("moe 1 token", 1, 7168, 2048, 32, 8),
        # a handful of requests; nearly every token has experts of its own
        _moe("moe 8 tokens", 8, 4096, 1536, 96, 8),
        # one rank's share of the experts (the others' slots are empty), odd block counts and batch
        _moe("moe 13 tokens, local half", 13, 2688, 896, 40, 6, local=0.5),
        # a full decode batch: every expert is hit, some by more than sixteen rows
        _moe("moe 64 tokens", 64, 7168, 2048, 64, 8),
        # sigmoid scores with a selection bias and expert groups, one token and a prefill
        _route("route 1 token", 1, 256, 8, "sigmoid", 8, 4, bias=True),
        _route("route 4096 tokens", 4096, 256, 8, "sigmoid", 8, 4, bias=True),
        # softmax scores of an odd number of experts, 16-bit logits (many ties), some experts switched off
        _route("route 333 tokens, 61 experts", 333, 61, 6, "softmax", dtype="bf16", masked=0.1),
        # before the attention or the experts of one token
        _norm("norm 1 token", 1, 7168, "block"),
        # norms on both sides of a block in a prefill
        _norm("norm 4096 tokens", 4096, 7168, "block", post=True),
        # per-token gate and residual scale, codes for the channel-wise layers, fp16
        _norm("norm 333 tokens, gated", 333, 4096, "token", dtype="fp16", post=True, gate="token", scale=0.22),
        # the norm in front of a layer that takes 16-bit inputs (a router, a head), per-channel gate, odd block count
        _norm("norm 1023 tokens, 16 bit", 1023, 2688, "normed", gate="channel", scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "route", "norm"])
    if op == "moe":
        while True:
            T, K, I = _log(rng, 1, 64), GROUP * _log(rng, 2, 64), GROUP * _log(rng, 1, 24)
            E = _log(rng, 4, 128)
            topk = rng.randint(1, min(8, E))
            # no more weights, and no more products, than the largest listed case
            if E * I * K <= 64 * 2048 * 7168 and T * topk <= 512:
                break
        return {"op": op, "T": T, "K": K, "I": I, "E": E, "topk": topk, "local": rng.choice([1.0, 1.0, 0.5])}
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 4, 384 // groups)
        kept = rng.randint((groups + 1) // 2, groups)
        topk = rng.randint(1, min(12, kept * (E // groups)))
        T = _log(rng, 1, min(4096, 4096 * 256 // E))
        return {"op": op, "T": T, "E": E, "topk": topk, "score": rng.choice(["softmax", "sigmoid"]), "groups": groups,
                "kept": kept, "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"]), "bias": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.0, 0.1])}
    K = GROUP * _log(rng, 2, 144)
    M = _log(rng, 1, min(4096, 4096 * 7168 // K))
    return {"op": op, "M": M, "K": K, "out": rng.choice(["block", "block", "token", "normed"]),
            "dtype": rng.choice(["bf16", "bf16", "fp16"]), "residual": rng.random() < 0.9, "post": rng.random() < 0.5,
            "gate": rng.choice(["none", "none", "channel", "token"]), "scale": rng.choice([1.0, 0.5, 0.22])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """N(0, 1) with about 0.5 % of the values 20 times as large."""
    x = _randn(g, M, K)
    far = torch.rand(M, K, generator=g, device="cuda") < 0.005
    return torch.where(far, x * 20, x)


def _group_quant(x):
    """The library's group quantiser of fp32 x [..., K]: integer-valued fp32 codes and scales."""
    v = x.reshape(*x.shape[:-1], -1, GROUP)
    s = v.abs().amax(-1).clamp_min(1e-10)
    s = s / torch.full_like(s, 127.0)
    return torch.round(v / s.unsqueeze(-1)).clamp(-127, 127).reshape(x.shape), s


def _weight_codes(g, E, N, K):
    w = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w[e:e + n] = _randn(g, n, N, K).mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    s = (0.75 + 0.5 * torch.rand(E, N // GROUP, K // GROUP, generator=g, device="cuda")) * (0.02 / 36.0)
    return w, s


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if case["op"] == "moe":
        T, K, I, E, k = case["T"], case["K"], case["I"], case["E"], case["topk"]
        q, sa = _group_quant(_activations(g, T, K))
        w13, s13 = _weight_codes(g, E, 2 * I, K)
        w2, s2 = _weight_codes(g, E, K, I)
        score, ids = torch.sigmoid(_randn(g, T, E)).topk(k, dim=1)
        wt = 2.5 * score / score.sum(1, keepdim=True)
        if case["local"] < 1.0:  # the slots of experts that another GPU holds
            ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < case["local"], ids, torch.full_like(ids, -1))
        c.update(A=q.to(torch.int8), sa=sa, w13=w13, s13=s13, w2=w2, s2=s2, ids=ids.to(torch.int32), wt=wt)
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = _randn(g, T, E) * 1.5
        if case["masked"]:
            logits = torch.where(torch.rand(T, E, generator=g, device="cuda") < case["masked"],
                                 torch.full_like(logits, -math.inf), logits)
        c.update(logits=logits.to(HALF[case["dtype"]]), corr=_randn(g, E) * 0.05 if case["bias"] else None)
    else:
        M, K, dt = case["M"], case["K"], HALF[case["dtype"]]
        gate = {"none": None, "channel": (K,), "token": (M, K)}[case["gate"]]
        c.update(y=(0.3 * _activations(g, M, K)).to(dt),
                 res=_activations(g, M, K).to(dt) if case["residual"] else None,
                 post_w=(1 + 0.2 * _randn(g, K)).to(dt) if case["post"] else None,
                 pre_w=(1 + 0.2 * _randn(g, K)).to(dt),
                 gate_v=None if gate is None else torch.sigmoid(_randn(g, *gate)).to(dt), eps=1e-6)
    return c


# ---------------------------------------------------------- the operators
def run(state):
    return {"moe": _run_moe, "route": _run_route, "norm": _run_norm}[state["op"]](state)


def _run_moe(c):
    if own:
        return _w8().moe_w8a8_block(c["A"], c["sa"], c["ids"], c["wt"], c["w13"], c["s13"], c["w2"], c["s2"])
    return _plain_moe(c["A"], c["sa"], c["ids"], c["wt"], c["w13"], c["s13"], c["w2"], c["s2"])


def _run_route(c):
    if own:
        w8 = _w8()
        return w8.moe_route_topk(c["logits"], c["topk"], bias=c["corr"],
                                 score=w8.W8_ROUTE_SIGMOID if c["score"] == "sigmoid" else w8.W8_ROUTE_SOFTMAX,
                                 n_group=c["groups"], topk_group=c["kept"], group_top=2, renormalise=True, scale=2.5)
    return _plain_route(c["logits"], c["corr"], c["topk"], c["score"], c["groups"], c["kept"])


def _run_norm(c):
    if own:
        w8 = _w8()
        scheme = {"block": w8.W8_SCHEME_BLOCK, "token": w8.W8_SCHEME_CHANNEL, "normed": None}[c["out"]]
        r = w8.norm_residual_quant(c["y"], c["pre_w"], residual=c["res"], post_weight=c["post_w"], gate=c["gate_v"],
                                   residual_scale=c["scale"], eps=c["eps"], scheme=scheme, normed=scheme is None)
        if scheme is None:
            return r
        h, q, s = r
        return h, _values(q, s, c["y"].dtype)
    return _plain_norm(c)


def _values(q, s, dtype):
    """What the codes stand for, in the activations' type."""
    M, K = q.shape
    v = torch.empty(M, s.numel() // M, s.numel() and M * K // s.numel(), dtype=dtype, device=q.device)
    return torch.mul(q.view(v.shape), s.reshape(M, -1, 1), out=v).view(M, K)


def _dequantised(w, s):
    E, N, K = w.shape
    v = w.view(E, N // GROUP, GROUP, K // GROUP, GROUP).float()
    return v.mul_(s[:, :, None, :, None]).view(E, N, K)


def _plain_moe(A, sa, ids, wt, w13, s13, w2, s2):
    T, K = A.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    x = (A.view(T, -1, GROUP).float() * sa.unsqueeze(-1)).view(T, K)
    there = (ids >= 0) & (ids < E)
    at = torch.where(there, ids, torch.zeros_like(ids)).long()
    wt = torch.where(there, wt, torch.zeros_like(wt))

    def act(gu):
        gate, up = gu[..., :I], gu[..., I:]
        h = gate / (1 + torch.exp(-gate)) * up
        q, s = _group_quant(h)
        return (q.view(*q.shape[:-1], -1, GROUP) * s.unsqueeze(-1)).view(q.shape)

    if ids.numel() <= E:  # each slot's own expert
        e = at.reshape(-1)
        xs = x.repeat_interleave(ids.shape[1], dim=0)
        h = act(torch.matmul(_dequantised(w13[e], s13[e]), xs.unsqueeze(-1)).squeeze(-1))
        o = torch.matmul(_dequantised(w2[e], s2[e]), h.unsqueeze(-1)).view(T, -1, K)
        return (o * wt.unsqueeze(-1)).sum(1).to(torch.bfloat16)
    # every expert on every token, and the weights of those that were chosen
    gu = torch.matmul(x, _dequantised(w13, s13).view(-1, K).t()).view(T, E, 2 * I)
    h = act(gu).transpose(0, 1).contiguous()
    o = torch.matmul(h, _dequantised(w2, s2).transpose(1, 2))
    share = torch.zeros(T, E, device=A.device).scatter_add_(1, at, wt)
    return (o * share.t().unsqueeze(-1)).sum(0).to(torch.bfloat16)


def _plain_route(logits, corr, topk, score, groups, kept):
    T, E = logits.shape
    l = logits.double()
    off = torch.isneginf(l) | torch.isnan(l)
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(-1e300))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    c = s + corr.double() if corr is not None else s
    c = torch.where(off, torch.full_like(c, -math.inf), c)
    if groups > 1:
        best = torch.sort(c.view(T, groups, -1), dim=2, descending=True).values[:, :, :2]
        second = torch.where(torch.isinf(best[..., 1:]), torch.zeros_like(best[..., 1:]), best[..., 1:])
        order = torch.sort(best[..., 0] + second.sum(-1), dim=1, descending=True, stable=True).indices[:, :kept]
        stays = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order, True)
        c = torch.where(stays.repeat_interleave(E // groups, dim=1), c, torch.full_like(c, -math.inf))
    c, ids = torch.sort(c, dim=1, descending=True, stable=True)
    c, ids = c[:, :topk], ids[:, :topk]
    w = torch.where(torch.isinf(c), torch.zeros_like(c), s.gather(1, ids))
    w = w / w.sum(1, keepdim=True).clamp_min(1e-300) * 2.5
    return torch.where(torch.isinf(c), torch.full_like(ids, -1), ids).to(torch.int32), w.float()


def _plain_norm(c):
    y, dt, K = c["y"].float(), c["y"].dtype, c["y"].shape[1]
    if c["post_w"] is not None:
        y = y * torch.rsqrt((y * y).sum(1, keepdim=True) / K + c["eps"]) * c["post_w"].float()
    if c["gate_v"] is not None:
        y = y * c["gate_v"].float()
    y = y * c["scale"]
    if c["res"] is not None:
        y = c["res"].float() + y
    h = y.to(dt)
    y = h.float()
    z = (y * torch.rsqrt((y * y).sum(1, keepdim=True) / K + c["eps"]) * c["pre_w"].float()).to(dt)
    if c["out"] == "normed":
        return h, z
    if c["out"] == "block":
        q, s = _group_quant(z.float())
    else:
        s = z.float().abs().amax(1, keepdim=True).clamp_min(1e-10)
        s = s / torch.full_like(s, 127.0)
        q = torch.round(z.float() / s).clamp(-127, 127)
    return h, _values(q, s, dt)


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = prepare(case, seed)
    return {"moe": _exact_moe, "route": _exact_route, "norm": _exact_norm}[case["op"]](c)


def _exact_codes(v):
    """Code times scale of the quantiser on 64-bit v [..., n]: the scale is an fp32 number by definition."""
    s = (v.abs().max(-1, keepdim=True).values.clamp(min=1e-10) / 127.0).float().double()
    return torch.clamp(torch.round((v / s).float().double()), -127, 127) * s


def _exact_moe(c):
    T, K = c["A"].shape
    I, E = c["I"], c["E"]
    x = c["A"].double() * c["sa"].double().repeat_interleave(GROUP, 1)
    out = torch.zeros(T, K, dtype=torch.float64, device=x.device)
    for e in range(E):
        t, j = torch.nonzero(c["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        w = c["w13"][e].double() * c["s13"][e].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        gu = torch.mm(x[t], w.t())
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        h = _exact_codes(h.view(-1, I // GROUP, GROUP)).view(-1, I)
        w = c["w2"][e].double() * c["s2"][e].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        out.index_add_(0, t, torch.mm(h, w.t()) * c["wt"][t, j].double().unsqueeze(1))
    return out


def _exact_route(c):
    import numpy as np
    l = c["logits"].double().cpu().numpy()
    T, E = l.shape
    off = ~(l > -np.inf)
    l = np.where(off, -np.inf, l)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-l))
    else:
        top = l.max(1, keepdims=True)
        e = np.where(off, 0.0, np.exp(l - np.where(np.isfinite(top), top, 0.0)))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    pick = np.where(off, -np.inf, s + (c["corr"].double().cpu().numpy() if c["corr"] is not None else 0.0))
    if c["groups"] > 1:
        v = np.sort(pick.reshape(T, c["groups"], -1), axis=2)[:, :, ::-1]
        score = v[:, :, 0] + np.where(np.isfinite(v[:, :, 1]), v[:, :, 1], 0.0)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1)
        pick = np.where(np.repeat(rank < c["kept"], E // c["groups"], axis=1), pick, -np.inf)
    ids = np.argsort(-pick, axis=1, kind="stable")[:, :c["topk"]]
    gone = np.isinf(np.take_along_axis(pick, ids, 1))
    w = np.where(gone, 0.0, np.take_along_axis(s, ids, 1))
    w = 2.5 * w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    return np.where(gone, -1, ids).astype(np.int32), w


def _exact_norm(c):
    y, dt = c["y"].double(), c["y"].dtype
    if c["post_w"] is not None:
        y = y / torch.sqrt(y.square().mean(1, keepdim=True) + c["eps"]) * c["post_w"].double()
    y = c["scale"] * y if c["gate_v"] is None else c["scale"] * c["gate_v"].double() * y
    h = y if c["res"] is None else y + c["res"].double()
    # the norm works on h as it is stored, the quantiser on the norm's 16-bit output
    y = h.to(dt).double()
    z = y / torch.sqrt(y.square().mean(1, keepdim=True) + c["eps"]) * c["pre_w"].double()
    if c["out"] == "normed":
        return h, z
    z = z.to(dt).double()
    if c["out"] == "token":
        return h, _exact_codes(z)
    return h, _exact_codes(z.view(z.shape[0], -1, GROUP)).view(z.shape)


# -------------------------------------------------------------------- work
def work(case):
    """Inputs read once, outputs written once; of the experts, those that T tokens are expected to choose."""
    if case["op"] == "moe":
        T, K, I, E, k = case["T"], case["K"], case["I"], case["E"], case["topk"]
        slots = T * k * case["local"]
        active = min(E * (1 - (1 - k / E * case["local"]) ** T), slots)
        return {"bytes": active * 3 * I * K * (1 + 4 / GROUP ** 2) + T * (K * (1 + 4 / GROUP + 2) + 8 * k),
                "flops": 6.0 * slots * I * K}
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        return {"bytes": T * E * (4 if case["dtype"] == "fp32" else 2) + 8 * T * case["topk"] + 4 * E,
                "flops": 4.0 * T * E}
    M, K = case["M"], case["K"]
    read = 2 * M * K * (1 + case["residual"] + (case["gate"] == "token"))
    read += 2 * K * (1 + case["post"] + (case["gate"] == "channel"))
    write = 2 * M * K + {"block": M * K + 4 * M * K // GROUP, "token": M * K + 4 * M, "normed": 2 * M * K}[case["out"]]
    return {"bytes": read + write, "flops": 12.0 * M * K}
