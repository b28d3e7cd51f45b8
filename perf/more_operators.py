"""The attention half of a decode step over a cache that is held in 4 or 8
bits, as a list of timed cases: keys and values quantised as they are written,
read back, and attention that reads the codes.

The cache is a tuple (k, k_scale, v, v_scale) of pages:
  k        [pages, heads, page, D / 2] uint8 (4 bits: channel 2j + 8 in the low
           nibble of byte j, 2j + 1 in the high one, offset by 8) or
           [pages, heads, page, D] int8
  v        [pages, heads, page / 4, 16, 4, Dv] of the same type: the D channels
           in sixteenths of Dv bytes, four tokens' sixteenths next to each other
  k_scale, v_scale   [pages, heads, page] fp32, one per token and head
A token's slot is page * page_size + its place in the page.

run(state) computes a case either in its plain form (elementary torch
operations in 32 bits) or, where `own` is true, through the library's entry
points quant_kv_cache, dequant_kv_cache and attn_kv_cache.  exact(case, seed)
is the definition in 64 bits.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _w8():
    import w8a8_int8_quantized_amd as w8
    return w8


# ------------------------------------------------------------------- cases
def _write(name, T, H, D, bits, page, dtype="bf16", padded=0.0):
    return {"name": name, "op": "write", "T": T, "H": H, "D": D, "bits": bits, "page": page, "dtype": dtype,
            "padded": padded}


def _read(name, T, H, D, bits, page, dtype="bf16"):
    return {"name": name, "op": "read", "T": T, "H": H, "D": D, "bits": bits, "page": page, "dtype": dtype}


def _attn(name, B, q, kv, Hq, Hkv, D, bits, page, dtype="bf16", spread=False, mixed=False, causal=True, lse=False):
    return {"name": name, "op": "attn", "B": B, "q": q, "kv": kv, "Hq": Hq, "Hkv": Hkv, "D": D, "bits": bits,
            "page": page, "dtype": dtype, "spread": spread, "mixed": mixed, "causal": causal, "lse": lse}


def listed():
    return [
        # one request being answered: its new key and value (latency counts)
        _write("write 1 token", 1, 8, 128, 4, 64),
        # a prompt of 4096 tokens
        _write("write 4096 tokens", 4096, 8, 128, 4, 64),
        # a padded batch, an odd number of heads, 8 bits
        _write("write 333 tokens, 8 bit", 333, 5, 64, 8, 16, dtype="fp16", padded=0.2),
        # a sequence's cache handed to 16-bit code: a long one, and a few tokens of wide heads
        _read("read 32768 tokens", 32768, 8, 128, 4, 64),
        _read("read 77 tokens, 8 bit", 77, 2, 256, 8, 32, dtype="fp16"),
        # one request, a short and a very long conversation
        _attn("attn 1 x 1000", 1, 1, 1000, 32, 8, 128, 4, 64),
        _attn("attn 1 x 131072", 1, 1, 131072, 32, 8, 128, 4, 64),
        # a full decode batch of requests of all lengths
        _attn("attn 64 x 16384, all lengths", 64, 1, 16384, 32, 8, 128, 4, 64, spread=True),
        # a key head per query head, odd batch and lengths, 8 bits, with the log of the sums for a later join
        _attn("attn 13 x 2501, 8 bit", 13, 1, 2501, 12, 12, 64, 8, 16, dtype="fp16", spread=True, lse=True),
        # four drafted tokens a request are verified, one key head for all query heads
        _attn("attn 7 x 4 drafted", 7, 4, 6007, 10, 1, 256, 4, 128, spread=True),
        # a step that mixes prompts' pieces with requests being answered, some places of the batch empty
        _attn("attn 24 mixed", 24, 700, 5000, 16, 4, 128, 4, 32, dtype="fp16", spread=True, mixed=True),
        # a piece of 2048 tokens of a long prompt
        _attn("attn 2048 of 8192", 1, 2048, 8192, 32, 8, 128, 4, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn"])
    bits, page = rng.choice([4, 4, 8]), rng.choice([16, 32, 48, 64, 128, 256])
    D, dtype = rng.choice([64, 128, 128, 256]), rng.choice(["bf16", "bf16", "fp16"])
    if op != "attn":
        H = _log(rng, 1, 16)
        T = _log(rng, 1, (4096 if op == "write" else 32768) * 1024 // (H * D))
        c = {"op": op, "T": T, "H": H, "D": D, "bits": bits, "page": page, "dtype": dtype}
        if op == "write":
            c["padded"] = rng.choice([0.0, 0.0, 0.2])
        elif rng.random() < 0.2:
            c["dtype"] = "fp32"
        return c
    while True:
        Hkv, G = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
        B, kv = _log(rng, 1, 64), _log(rng, 1, 131072)
        q = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 8, 2048)])
        spread = rng.random() < 0.6
        # no more of the cache, and no more products, than the largest listed cases
        if (q <= kv and Hkv * G <= 64 and B * kv * Hkv * D <= 64 * 8192 * 8 * 128 and kv * Hkv * D <= 1 << 27
                and B * q * kv * Hkv * G * D <= 2048 * 8192 * 32 * 128):
            break
    return {"op": op, "B": B, "q": q, "kv": kv, "Hq": Hkv * G, "Hkv": Hkv, "D": D, "bits": bits, "page": page,
            "dtype": dtype, "spread": spread, "mixed": spread and q > 1 and rng.random() < 0.5,
            "causal": rng.random() < 0.8, "lse": rng.random() < 0.3}


def _lengths(c):
    """Each sequence's query and cached tokens (the queries' own among them): of the case, not of the seed."""
    rng = random.Random(1000003 * c["B"] + 1009 * c["kv"] + c["q"])
    out = []
    for b in range(c["B"]):
        q, kv = c["q"], c["kv"]
        if b and c["spread"]:
            kv = rng.randint(q if not c["mixed"] else 1, kv)
            if c["mixed"]:
                q = 1 if rng.random() < 0.7 else rng.randint(1, min(q, kv))
            if b % 8 == 5:  # a place of the batch without a request
                q, kv = 1, 0
        out.append((q, kv))
    return out


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(g, *shape):
    """Keys or values: N(0, 1) with a few channels four times as large."""
    far = torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.04, 4.0, 1.0)
    return _randn(g, *shape) * far


def _pack(codes, bits):
    """Integer-valued codes [..., D] as the cache's bytes."""
    if bits == 8:
        return codes.to(torch.int8)
    u = (codes + 8).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _unpack(b):
    """The codes of the cache's bytes, fp32 [..., D]."""
    if b.dtype == torch.int8:
        return b.float()
    return torch.stack((b & 15, b >> 4), -1).flatten(-2).float() - 8


def _fours(b):
    """Bytes [..., page, Db] of value rows in the cache's order, and
    _straight back."""
    s = b.shape
    return b.view(*s[:-2], s[-2] // 4, 4, 16, s[-1] // 16).transpose(-2, -3).contiguous()


def _straight(b):
    s = b.shape
    return b.transpose(-2, -3).reshape(*s[:-4], s[-4] * 4, 16 * s[-1])


def _cache(g, pages, H, page, D, bits):
    """A cache whose every slot is written: codes and scales of rows as _rows gives them."""
    top = 7.0 if bits == 4 else 127.0
    out = []
    for is_v in (False, True):
        codes = torch.empty(pages, H, page, D * bits // 8, dtype=torch.uint8 if bits == 4 else torch.int8,
                            device="cuda")
        step = max(1, (1 << 26) // (H * page * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            codes[p:p + n] = _pack(_rows(g, n, H, page, D).mul_(top / 3.0).round_().clamp_(-top, top), bits)
        scale = (0.6 + 0.8 * torch.rand(pages, H, page, generator=g, device="cuda")) * (3.0 / top)
        out += [_fours(codes) if is_v else codes, scale]
    return tuple(out)


def _slots(g, T, pages, page):
    """T tokens of sequences whose pages lie anywhere: slots in order within a page."""
    at = torch.randperm(pages, generator=g, device="cuda")
    s = (at.unsqueeze(1) * page + torch.arange(page, device="cuda")).flatten()
    return s[:T].to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    D, bits, page, dt = c["D"], c["bits"], c["page"], TYPES[c["dtype"]]
    if c["op"] != "attn":
        T, H = c["T"], c["H"]
        pages = (T + page - 1) // page + 3
        c.update(cache=_cache(g, pages, H, page, D, bits), slots=_slots(g, T, pages, page))
        if c["op"] == "write":
            # the two lie in the output of one projection, next to each other
            kv = _rows(g, T, 2, H, D).to(dt)
            c.update(kn=kv[:, 0], vn=kv[:, 1])
            if c["padded"]:
                c["slots"] = torch.where(torch.rand(T, generator=g, device="cuda") < c["padded"],
                                         torch.full_like(c["slots"], -1), c["slots"])
        return c
    c["lens"] = lens = _lengths(c)
    per = [(kv + page - 1) // page for _, kv in lens]
    pages = sum(per) + 2
    c["cache"] = _cache(g, pages, c["Hkv"], page, D, bits)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["B"], max(per)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for q, _ in lens:
        starts.append(starts[-1] + q)
    c.update(table=table, kv_lens=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
             starts=starts, q_starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
             # queries somewhat larger than 1, so that some tokens are attended to more than others
             x=(1.5 * _randn(g, starts[-1], c["Hq"], D)).to(dt))
    return c


# ---------------------------------------------------------- the operators
def run(state):
    return {"write": _run_write, "read": _run_read, "attn": _run_attn}[state["op"]](state)


def _run_write(c):
    """The rows are written, and what the cache now holds of them is read back."""
    if own:
        w8 = _w8()
        w8.quant_kv_cache(c["kn"], c["vn"], c["slots"], c["cache"])
        return w8.dequant_kv_cache(c["cache"], c["slots"], dtype=c["kn"].dtype)
    _plain_write(c["kn"], c["vn"], c["slots"], c["cache"], c["bits"], c["page"])
    return _plain_read(c["cache"], c["slots"], c["page"], c["kn"].dtype)


def _run_read(c):
    if own:
        return _w8().dequant_kv_cache(c["cache"], c["slots"], dtype=TYPES[c["dtype"]])
    return _plain_read(c["cache"], c["slots"], c["page"], TYPES[c["dtype"]])


def _run_attn(c):
    if own:
        ragged = {} if not c["spread"] else {"q_starts": c["q_starts"], "max_q": c["q"]}
        return _w8().attn_kv_cache(c["x"], c["cache"], c["table"], c["kv_lens"], causal=c["causal"], lse=c["lse"],
                                   **ragged)
    return _plain_attn(c)


def _plain_write(kn, vn, slots, cache, bits, page):
    k, ks, v, vs = cache
    live = slots >= 0
    s = slots[live].long()
    p, o = s // page, s % page
    top = 7.0 if bits == 4 else 127.0
    for x, is_v in ((kn, False), (vn, True)):
        x = x[live].float()
        scale = x.abs().amax(-1).clamp_min(1e-10)
        scale = scale / torch.full_like(scale, top)
        b = _pack(torch.round(x / scale.unsqueeze(-1)).clamp(-top, top), bits)
        if is_v:
            v[p, :, o // 4, :, o % 4] = b.view(*b.shape[:2], 16, -1)
            vs[p, :, o] = scale
        else:
            k[p, :, o] = b
            ks[p, :, o] = scale


def _plain_read(cache, slots, page, dt):
    k, ks, v, vs = cache
    live = (slots >= 0).view(-1, 1, 1)
    s = slots.clamp_min(0).long()
    p, o = s // page, s % page
    kr = _unpack(k[p, :, o]) * ks[p, :, o].unsqueeze(-1)
    vr = _unpack(v[p, :, o // 4, :, o % 4].flatten(-2)) * vs[p, :, o].unsqueeze(-1)
    return tuple(torch.where(live, r, torch.zeros_like(r)).to(dt) for r in (kr, vr))


def _plain_attn(c):
    x, (k, ks, v, vs) = c["x"], c["cache"]
    B, n, Hq, Hkv, D = c["B"], c["q"], c["Hq"], c["Hkv"], c["D"]
    G, L = Hq // Hkv, c["table"].shape[1] * c["page"]
    at = c["table"].clamp_min(0).long()
    kb = (_unpack(k[at]) * ks[at].unsqueeze(-1)).transpose(1, 2).reshape(B * Hkv, L, D)
    vb = (_unpack(_straight(v[at])) * vs[at].unsqueeze(-1)).transpose(1, 2).reshape(B * Hkv, L, D)
    # every sequence's queries in n places, and the last key that each of them sees
    first, last = c["q_starts"][:-1].long().view(B, 1), c["q_starts"][1:].long().view(B, 1)
    rows = first + torch.arange(n, device=x.device)
    there = rows < last
    rows = torch.where(there, rows, torch.zeros_like(rows))
    seen = c["kv_lens"].view(B, 1) + torch.arange(1, n + 1, device=x.device) - (last - first) if c["causal"] \
        else c["kv_lens"].view(B, 1).expand(B, n)
    hidden = torch.arange(L, device=x.device).view(1, 1, L) >= seen.repeat_interleave(G, dim=1).unsqueeze(-1)
    xb = x[rows].float().view(B, n, Hkv, G, D).transpose(1, 2).reshape(B * Hkv, n * G, D)
    s = torch.matmul(xb, kb.transpose(1, 2).contiguous()).view(B, Hkv, n * G, L) * D ** -0.5
    s = torch.where(hidden.unsqueeze(1), torch.full((), -math.inf, device=x.device), s)
    m = s.amax(-1, keepdim=True)
    s = torch.exp(s - m.clamp_min(-3e38))
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B * Hkv, n * G, L), vb).view(B, Hkv, n * G, D) / total.clamp_min(1e-30)
    o = o.view(B, Hkv, n, G, D).transpose(1, 2).reshape(B, n, Hq, D)[there].to(x.dtype)
    if not c["lse"]:
        return o
    return o, (m + torch.log(total)).view(B, Hkv, n, G).transpose(1, 2).reshape(B, n, Hq)[there]


# ------------------------------------------------- the definition in 64 bits
def _nibbles(b):
    """Codes of packed or plain bytes [..., n] as fp64."""
    if b.dtype == torch.int8:
        return b.double()
    out = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.float64, device=b.device)
    out[..., 0::2] = (b % 16).double()
    out[..., 1::2] = torch.div(b, 16, rounding_mode="floor").double()
    return out - 8.0


def exact(case, seed):
    c = prepare(case, seed)
    if case["op"] == "write":
        top = 7.0 if case["bits"] == 4 else 127.0
        live = (c["slots"] >= 0).double().view(-1, 1, 1)
        out = []
        for x in (c["kn"].double(), c["vn"].double()):
            # the scale is an fp32 number, and a code the nearest integer of an fp32 quotient, by definition
            s = (x.abs().max(-1, keepdim=True).values.clamp(min=1e-10) / top).float().double()
            out.append(torch.clamp(torch.round((x / s).float().double()), -top, top) * s * live)
        return tuple(out)
    k, ks, v, vs = c["cache"]
    page, D = case["page"], case["D"]
    if case["op"] == "read":
        s = c["slots"].long()
        p, o = torch.div(s, page, rounding_mode="floor"), torch.remainder(s, page)
        q = torch.div(o, 4, rounding_mode="floor")
        kr = _nibbles(k[p, :, o]) * ks[p, :, o].double()[..., None]
        vr = torch.cat([_nibbles(v[p, :, q, i, o - 4 * q]) for i in range(16)], -1) * vs[p, :, o].double()[..., None]
        return kr, vr
    T, Hq, Hkv = c["x"].shape[0], case["Hq"], case["Hkv"]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(c["lens"]):
        if n == 0 or L == 0:
            continue
        t0 = c["starts"][b]
        at = torch.arange(L, device="cuda")
        p = c["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
        o = at % page
        hidden = None
        if case["causal"]:
            hidden = at.view(1, L) > torch.arange(n, device="cuda").view(n, 1) + (L - n)
        for h in range(Hkv):
            kh = _nibbles(k[p, h, o]) * ks[p, h, o].double().view(L, 1)
            vh = torch.cat([_nibbles(v[p, h, o // 4, i, o % 4]) for i in range(16)], 1) * vs[p, h, o].double().view(L, 1)
            for j in range(h * G, h * G + G):
                s = torch.mm(c["x"][t0:t0 + n, j].double(), kh.t()) / math.sqrt(D)
                if hidden is not None:
                    s = s.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(s, 1)
                out[t0:t0 + n, j] = torch.mm(torch.exp(s - z.view(n, 1)), vh)
                lse[t0:t0 + n, j] = z
    return (out, lse) if case["lse"] else out


# -------------------------------------------------------------------- work
def work(case):
    """Inputs read once, outputs and what the cache gains written once; of the cache, the tokens that are attended to."""
    D, row = case["D"], case["D"] * case["bits"] / 8 + 4
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] != "attn":
        n = case["T"] * case["H"] * 2
        if case["op"] == "write":
            return {"bytes": n * (2 * D * size + row) + 4 * case["T"], "flops": 4.0 * n * D}
        return {"bytes": n * (D * size + row) + 4 * case["T"], "flops": 1.0 * n * D}
    b = f = 0.0
    for q, kv in _lengths(case):
        pairs = q * kv - (q * (q - 1) / 2 if case["causal"] else 0)
        b += 2 * kv * case["Hkv"] * row + 2 * q * case["Hq"] * D * size + 4 * q * case["Hq"] * case["lse"]
        f += 4.0 * pairs * case["Hq"] * D
    return {"bytes": b, "flops": f}
