"""GPU parity of the quantised key/value cache and the attention over it
against the 64-bit oracle (oracle/cache.py).

Tolerances, each derived before the first run (u32 = 2^-24, half a step of
fp32; u16 = 2^-11, of fp16):
  write  codes and scales are the oracle's, bit for bit.
  read   code times scale in fp32, rounded once: the oracle's, bit for bit.
  attention
    score  a sum of D exact products and a starting value, fp32, in an order
           that is not ours: D + 1 additions of a partial sum of at most
           offset (sum |q| + |sum q|) + 127 sum |q| in codes, whose
           roundings have either sign; six standard deviations of such a sum
           are 6 sqrt(D + 1) u32 of it (offset: at most 1152, in which a code
           is held).  Times the token's scale and the call's, two products
           more (4 u32 of the score), and the exponent's own rounding, of a
           number of up to |s| + |m|, with 2 units of the instruction: per
           token 6 sqrt(D + 1) u32 codes scale ks + u32 (5 |s| + |m| + 4).
           What that moves at most is the oracle's.
    sums   p vs in fp16: u16, and what is below its normal range 2^-35 of the
           largest term at most; sums of n terms, at most n / 32 + 8
           sequential additions and 32 inside an instruction: (n / 32 + 40) u32.
    out    the scores' part; u16 + 2 sums of mag = sum p |v| / sum p; n 2^-35
           127 max vs; the output's rounding.
    lse    the scores' part + the sums' + 4 u32 (|lse| + 1).
"""

import math

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_amd as w8
from oracle import cache as oc
from oracle import formats

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _np(t):
    """fp16 and fp32 as they are, bf16 as bits."""
    t = t.detach().cpu().contiguous()
    return t.view(torch.int16).numpy().view(np.uint16) if t.dtype == BF else t.numpy()


def _f64(t):
    return t.detach().cpu().double().numpy()


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _same(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


def _empty_np(pages, H, page, D, bits, seed):
    """Arrays of a cache that was used before: any bytes, scales NaN and infinite among them."""
    rng = np.random.default_rng(seed)
    db = D * bits // 8
    junk = np.array([np.nan, np.inf, -np.inf, 1e30, -1.0, 0.0], np.float32)
    return (rng.integers(0, 256, (pages, H, page, db), np.uint8), junk[rng.integers(0, 6, (pages, H, page))],
            rng.integers(0, 256, (pages, H, page // 4, 16, 4, db // 16), np.uint8),
            junk[rng.integers(0, 6, (pages, H, page))])


def _to_gpu(c, bits):
    dt = torch.uint8 if bits == 4 else torch.int8
    return tuple(torch.from_numpy(x).view(dt).to(DEV) if x.dtype == np.uint8 else torch.from_numpy(x).to(DEV)
                 for x in c)


# ------------------------------------------------------------ write and read
WRITES = [(1, 1, 64, 4, 16), (1, 8, 128, 4, 64), (3, 2, 256, 4, 16), (7, 5, 64, 8, 48), (33, 3, 128, 8, 16),
          (18, 1, 256, 8, 32), (130, 4, 128, 4, 32), (67, 12, 64, 4, 128)]


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("T,H,D,bits,page", WRITES)
def test_write_and_read(T, H, D, bits, page, dt):
    print(f"write T={T} H={H} D={D} bits={bits} page={page} {dt}", flush=True)
    g = _gen(T * 131 + D)
    pages = T // page + 3
    kv = torch.randn(T, 2, H, D, generator=g) * torch.exp(2 * torch.randn(T, 2, H, 1, generator=g))
    kv[0, 0, 0] = 0                                        # a row of zeros
    kv[0, 1, H - 1] = 3.5 * torch.sign(torch.randn(D, generator=g))
    if T > 2:
        kv[1] *= 1e-7 if dt == FP else 1e-30               # below the quantiser's floor
        kv[2, 0, 0, :15] = torch.arange(-7, 8) + 0.5       # halves: round to even
        kv[2, 0, 0, 15:] = 0
        kv[2, 0, 0, 20] = 7 if bits == 4 else 127
    kv = kv.to(dt)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[4], slots[3] = -1, pages * page              # padding, and past the end
    before = _empty_np(pages, H, page, D, bits, T)
    c = _to_gpu(before, bits)
    x = kv.to(DEV)
    w8.quant_kv_cache(x[:, 0], x[:, 1], slots.to(DEV), c)
    want = tuple(a.copy() for a in before)
    kq, ks = oc.quant_rows(_np(kv[:, 0]), bits)
    vq, vs = oc.quant_rows(_np(kv[:, 1]), bits)
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < pages * page:
            for h in range(H):
                oc.put(want, s // page, s % page, h, kq[t, h], ks[t, h], vq[t, h], vs[t, h], bits)
    for name, a, b in zip(("k", "k_scale", "v", "v_scale"), c, want):
        a = a.cpu().numpy()
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8)), name   # every other byte as it was
    # back, a slot twice, one that is nowhere and one past the end
    ask = torch.cat([slots, slots[:1], torch.tensor([-5, pages * page, 2 ** 31 - 1], dtype=torch.int32)])
    n = ask.numel()
    ok = ((ask >= 0) & (ask < pages * page)).numpy()
    for odt in (BF, FP, torch.float32):
        got = w8.dequant_kv_cache(c, ask.to(DEV), dtype=odt)
        for o, q, s in zip(got, (kq, vq), (ks, vs)):
            r = np.zeros((n, H, D), np.float32)
            r[:T + 1] = np.concatenate([q, q[:1]]).astype(np.float32) * np.concatenate([s, s[:1]])[..., None]
            r[~ok] = 0
            with np.errstate(over="ignore"):
                e = formats.f32_to_bf16_bits(r) if odt == BF else r.astype(np.float16) if odt == FP else r
            # (-0 and 0: a zero code times a scale)
            assert np.array_equal(_np(o).view(np.uint16 if odt != torch.float32 else np.uint32),
                                  e.view(np.uint16 if odt != torch.float32 else np.uint32)), odt


def test_write_rows_as_they_lie_in_a_projection():
    """Strided rows of a fused projection, an out-of-order batch over page borders."""
    T, Hq, H, D, page = 45, 8, 2, 128, 16
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=_gen(0), dtype=torch.float32).to(BF).to(DEV)
    k = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D)
    v = qkv[:, (Hq + H) * D:].view(T, H, D)
    slots = (torch.arange(T, dtype=torch.int32) + 9).flip(0).contiguous().to(DEV)
    a = _to_gpu(_empty_np(4, H, page, D, 4, 1), 4)
    b = tuple(t.clone() for t in a)
    w8.quant_kv_cache(k, v, slots, a)
    w8.quant_kv_cache(k.contiguous(), v.contiguous(), slots, b)
    assert _same(a, b)
    got = w8.dequant_kv_cache(a, slots, dtype=torch.float32)
    q, s = oc.quant_rows(_np(k), 4)
    assert np.array_equal(got[0].cpu().numpy(), q.astype(np.float32) * s[..., None])


def test_group_quantisers_give_the_same_rows():
    """128 channels: codes and scales of quant_act_group and quant_weight_int4_group."""
    T, H = 21, 3
    x = torch.randn(T, H, 128, generator=_gen(5)).to(FP).to(DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    for bits, fn in ((8, w8.quant_act_group), (4, w8.quant_weight_int4_group)):
        c = w8.kv_cache_empty(2, H, 16, 128, bits=bits)
        w8.quant_kv_cache(x, x, slots, c)
        q, s = fn(x.view(T * H, 128))
        k = c[0].transpose(1, 2).reshape(32, H, -1)[:T].reshape(T * H, -1)
        assert torch.equal(k, q) and torch.equal(c[1].transpose(1, 2).reshape(32, H)[:T].reshape(-1), s.view(-1))


def test_write_empty_and_refusals():
    c = w8.kv_cache_empty(2, 3, 16, 64)
    x = torch.zeros(4, 3, 64, dtype=BF, device=DEV)
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    w8.quant_kv_cache(x[:0], x[:0], i[:0], c)
    assert w8.dequant_kv_cache(c, i[:0])[0].shape == (0, 3, 64)
    for bad in [lambda: w8.quant_kv_cache(x[:, :2], x[:, :2], i, c), lambda: w8.quant_kv_cache(x.float(), x.float(), i, c),
                lambda: w8.quant_kv_cache(x, x.to(FP), i, c), lambda: w8.quant_kv_cache(x, x, i.long(), c),
                lambda: w8.quant_kv_cache(x, x, i[:3], c), lambda: w8.quant_kv_cache(x.transpose(0, 1), x, i, c),
                lambda: w8.quant_kv_cache(x, x, i, (c[0], c[1], c[2].view(-1), c[3])),
                lambda: w8.quant_kv_cache(x, x, i, (c[0], c[1].half(), c[2], c[3])),
                lambda: w8.quant_kv_cache(x, x, i, (c[0].float(), c[1], c[2], c[3])),
                lambda: w8.quant_kv_cache(torch.zeros(4, 64, 3, dtype=BF, device=DEV).transpose(1, 2), x, i, c),
                lambda: w8.dequant_kv_cache(c, i.view(2, 2)), lambda: w8.dequant_kv_cache(c, i, dtype=torch.float64),
                lambda: w8.dequant_kv_cache(c, i, out=(x, x.float()))]:
        with pytest.raises(w8.W8Error):
            bad()


# ---------------------------------------------------------------- attention
class Problem:
    """Sequences of (query tokens, cached tokens) over a cache whose other slots hold anything."""

    def __init__(self, lens, Hq, Hkv, D, bits, page, dt, seed=0, q_scale=1.5, spread=0.0, spare=1, first_row=0,
                 behind=0):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.bits, self.page, self.dt = lens, Hq, Hkv, D, bits, page, dt
        per = [-(-L // page) for _, L in lens]
        pages = sum(per) + 1
        c = _empty_np(pages, Hkv, page, D, bits, seed)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(per + [0]) + spare), -7, np.int32)
        self.k, self.ks, self.v, at = [], [], [], 0
        for b, (n, L) in enumerate(lens):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            rows = []
            for _ in range(2):
                x = rng.normal(size=(L, Hkv, D)) * np.exp(spread * rng.normal(size=(L, Hkv, 1)))
                rows.append(oc.quant_rows(x.astype(np.float32), bits))
            (kq, ks), (vq, vs) = rows
            for t in range(L):
                for h in range(Hkv):
                    oc.put(c, self.table[b, t // page], t % page, h, kq[t, h], ks[t, h], vq[t, h], vs[t, h], bits)
            self.k.append(kq * ks[..., None].astype(np.float64))
            self.ks.append(ks.astype(np.float64))
            self.v.append(vq * vs[..., None].astype(np.float64))
            self.vs_max = max(getattr(self, "vs_max", 0.0), float(vs.max(initial=0)))
        self.starts = np.cumsum([first_row] + [n for n, _ in lens]).astype(np.int32)
        T = int(self.starts[-1]) + behind
        self.q = (q_scale * torch.from_numpy(rng.normal(size=(T, Hq, D)))).to(dt)
        self.cache = _to_gpu(c, bits)

    def call(self, ragged=True, q=None, table=None, lens=None, **kw):
        i32 = {"dtype": torch.int32, "device": DEV}
        if ragged:
            kw.setdefault("q_starts", torch.tensor(self.starts, **i32))
            kw.setdefault("max_q", max([n for n, _ in self.lens] + [1]))
        return w8.attn_kv_cache(self.q.to(DEV) if q is None else q, self.cache,
                                torch.tensor(self.table, **i32) if table is None else table,
                                torch.tensor([L for _, L in self.lens], **i32) if lens is None else lens, **kw)

    def check(self, out, lse=None, scale=None, causal=True, only=None, sample=None):
        """sample: that many queries of each sequence, the first and the last among them."""
        scale = self.D ** -0.5 if scale is None else scale
        half = torch.finfo(self.dt).eps / 2
        tiny = torch.finfo(self.dt).smallest_normal * half
        o, z, q = _f64(out), None if lse is None else _f64(lse), _f64(self.q)
        worst = 0.0
        for b, (n, L) in enumerate(self.lens):
            if only is not None and b not in only:
                continue
            at = slice(int(self.starts[b]), int(self.starts[b]) + n)
            qa = np.abs(q[at]).sum(-1)
            codes = 1152 * (qa + np.abs(q[at].sum(-1))) + 127 * qa                        # [n, Hq]

            def score_error(i, j, x):
                ks = self.ks[b][:len(x), j // (self.Hq // self.Hkv)]
                return (6 * math.sqrt(self.D + 1) * U32 * codes[i, j] * abs(scale) * ks
                        + U32 * (5 * np.abs(x) + np.abs(x).max() + 4))

            which = range(n) if sample is None or n <= sample else sorted(
                {0, n - 1} | set(np.random.default_rng(n).integers(0, n, sample - 2).tolist()))
            ro, rz, mag, out_off, lse_off = oc.attention(q[at], self.k[b], self.v[b], scale, causal, score_error, which)
            sums = (L / 32 + 40) * U32
            e = out_off + (2.0 ** -11 + 2 * sums) * mag + L * 2.0 ** -35 * 127 * self.vs_max
            bound = half * (np.abs(ro) + e) + e + tiny
            assert np.isfinite(o[at]).all()
            d = np.zeros_like(ro)
            d[which] = np.abs(o[at] - ro)[which]
            worst = max(worst, float((d / bound).max(initial=0)))
            assert (d <= bound).all(), (b, float((d / bound).max()))
            if z is not None:
                zb, rz, lse_off = z[at][which], rz[which], lse_off[which]
                empty = np.isneginf(rz)
                assert np.array_equal(np.isneginf(zb), empty)
                bz = lse_off + sums + 4 * U32 * (np.abs(np.where(empty, 0, rz)) + 1)
                dz = np.abs(np.where(empty, 0, zb) - np.where(empty, 0, rz))
                assert (dz <= bz).all(), (b, float((dz / bz).max()))
        return worst


FORMS = [(64, 4), (128, 4), (256, 4), (64, 8), (128, 8), (256, 8)]
# A block table that is wider than short segments may be: they are shared out
# over workgroups then, and each by a workgroup of its own otherwise.
WIDE = 2000
LENGTHS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 130, 257]


@pytest.mark.parametrize("spare", [1, WIDE])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
def test_single_tokens_of_every_length(D, bits, dt, spare):
    print(f"attn lengths D={D} bits={bits} {dt} spare={spare}", flush=True)
    p = Problem([(1, L) for L in LENGTHS] + [(1, 0)], 6, 2, D, bits, 16, dt, seed=D + bits, spare=spare)
    out, lse = p.call(ragged=False, lse=True)
    print("share of the tolerance", p.check(out, lse))
    assert not out[-1].any() and torch.isneginf(lse[-1]).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (4, 2), (24, 3), (17, 1), (40, 1)])
@pytest.mark.parametrize("D,bits", [(64, 4), (128, 4), (256, 4), (128, 8)])
@pytest.mark.parametrize("spare", [1, WIDE])
def test_head_layouts_and_query_tokens(D, bits, Hq, Hkv, causal, spare):
    print(f"attn heads {Hq}/{Hkv} D={D} bits={bits} causal={causal} spare={spare}", flush=True)
    lens = [(3, 40), (1, 77), (0, 50), (9, 9), (6, 2), (1, 0), (4, 0), (20, 133)]
    p = Problem(lens, Hq, Hkv, D, bits, 32, BF if Hq % 2 else FP, seed=Hq, first_row=2, behind=3,
                spare=spare)
    i32 = p.q.shape[0], Hq
    out = torch.full((*i32, D), 7.5, dtype=p.dt, device=DEV)
    lse = torch.full(i32, 7.5, device=DEV)
    p.call(causal=causal, lse=True, out=(out, lse))
    p.check(out, lse, causal=causal)
    for t in (out, lse):      # rows of no sequence
        assert (t[:2] == 7.5).all() and (t[-3:] == 7.5).all()


@pytest.mark.parametrize("page", [16, 48, 80, 256])
@pytest.mark.parametrize("bits", [4, 8])
def test_pages_and_splits(page, bits):
    """Lengths that many workgroups share, in pages that end inside a tile."""
    print(f"attn pages {page} bits={bits}", flush=True)
    p = Problem([(1, 2500), (2, 31), (1, 1999), (1, 3)], 8, 2, 128, bits, page, BF, seed=page)
    out, lse = p.call(lse=True)
    print("share of the tolerance", p.check(out, lse))


@pytest.mark.parametrize("D,bits,n,L,Hq,Hkv", [(128, 4, 70, 300, 8, 2), (64, 8, 129, 129, 3, 3), (256, 4, 33, 200, 4, 1),
                                                (128, 8, 50, 1000, 4, 4), (64, 4, 257, 400, 2, 1)])
def test_pieces_of_prompts(D, bits, n, L, Hq, Hkv):
    print(f"attn prompt n={n} L={L} {Hq}/{Hkv} D={D} bits={bits}", flush=True)
    p = Problem([(n, L), (1, L - 1)], Hq, Hkv, D, bits, 16, FP, seed=n)
    out, lse = p.call(lse=True)
    print("share of the tolerance", p.check(out, lse))


# T * Hq query rows pick the row tile: 16 up to 4096 rows, 32 up to 40000, 64
# from there on (256 channels: 16), where a sequence has more than 16.
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,bits", FORMS)
def test_row_tiles_of_32(D, bits, causal, dt):
    print(f"attn 32 rows D={D} bits={bits} causal={causal} {dt}", flush=True)
    p = Problem([(400, 411), (1, 700), (150, 97), (0, 5), (3, 0)], 8, 2, D, bits, 48, dt, seed=D)
    assert p.q.shape[0] * 8 >= 4096
    out, lse = p.call(lse=True, causal=causal)
    print("share of the tolerance", p.check(out, lse, causal=causal, sample=12))


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits,Hq,Hkv", [(64, 4, 10, 2), (128, 4, 32, 8), (256, 4, 4, 1), (64, 8, 6, 6), (128, 8, 20, 4),
                                            (256, 8, 9, 1), (128, 4, 33, 1)])
def test_row_tiles_of_64(D, bits, Hq, Hkv, dt):
    print(f"attn 64 rows D={D} bits={bits} {Hq}/{Hkv} {dt}", flush=True)
    n = 40000 // Hq
    p = Problem([(n - 200, 301), (1, 900), (150, 450), (0, 9), (77, 77)], Hq, Hkv, D, bits, 64, dt, seed=Hq, behind=25)
    assert p.q.shape[0] * Hq >= 40000
    out, lse = p.call(lse=True)
    print("share of the tolerance", p.check(out, lse, sample=10))
    # scores that rise by hundreds
    p.q = (20 * p.q.float()).to(dt)
    out, lse = p.call(lse=True, causal=False)
    p.check(out, lse, causal=False, sample=10)


def test_more_sequences_than_threads():
    rng = np.random.default_rng(8)
    lens = [(int(rng.integers(0, 4)), int(rng.integers(0, 70))) for _ in range(700)]
    p = Problem(lens, 4, 2, 64, 4, 16, BF, seed=9)
    out, lse = p.call(lse=True)
    p.check(out, lse)


@pytest.mark.parametrize("bits", [4, 8])
def test_cache_beyond_four_gigabytes(bits):
    """Slots whose bytes lie past 32 bits, written, read back and attended to."""
    H, D, page = 4, 128, 256
    pages = (5 << 30) // (H * page * D * bits // 8)
    c = w8.kv_cache_empty(pages, H, page, D, bits=bits)
    assert c[0].numel() > 1 << 32
    L = 600
    kv = torch.randn(L, 2, H, D, generator=_gen(bits)).to(BF)
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    pos = torch.arange(L, device=DEV)
    slots = (table[0, pos // page] * page + pos % page).to(torch.int32)
    x = kv.to(DEV)
    w8.quant_kv_cache(x[:, 0], x[:, 1], slots, c)
    got = w8.dequant_kv_cache(c, slots, dtype=torch.float32)
    p = Problem([(1, 0)], 8, H, D, bits, page, BF, seed=3)
    p.lens, rows = [(1, L)], []
    for i in range(2):
        q, s = oc.quant_rows(_np(kv[:, i]), bits)
        assert np.array_equal(got[i].cpu().numpy(), q.astype(np.float32) * s[..., None])
        rows.append((q * s[..., None].astype(np.float64), s.astype(np.float64)))
    (k, ks), (v, vs) = rows
    p.k, p.ks, p.v, p.vs_max = [k], [ks], [v], float(vs.max())
    p.check(w8.attn_kv_cache(p.q.to(DEV), c, table, torch.tensor([L], dtype=torch.int32, device=DEV)))


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own, the same cache read by both."""
    p = Problem([(1, 5000), (1, 300), (1, 2222)], 8, 2, 128, 4, 64, BF, seed=12, spare=WIDE)
    i32 = {"dtype": torch.int32, "device": DEV}
    args = (p.q.to(DEV), p.cache, torch.tensor(p.table, **i32), torch.tensor([L for _, L in p.lens], **i32))
    want = w8.attn_kv_cache(*args, lse=True)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for i, s in enumerate(side):
            with torch.cuda.stream(s):
                outs[i].append(w8.attn_kv_cache(*args, lse=True))
    torch.cuda.synchronize()
    assert all(_same(want, o) for o in outs[0] + outs[1])


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    D, bits = FORMS[int(rng.integers(0, 6))]
    Hkv, G = int(rng.integers(1, 5)), int(rng.integers(1, 12))
    page = 16 * int(rng.integers(1, 9))
    lens = []
    for _ in range(int(rng.integers(1, 7))):
        L = int(np.exp(rng.uniform(0, np.log(1500))))
        lens.append((int(rng.integers(0, 1 + min(L, 30))) if rng.random() < 0.5 else 1, L))
    causal, dt = bool(rng.integers(0, 2)), (BF, FP)[int(rng.integers(0, 2))]
    print(f"attn drawn {lens} {Hkv}x{G} D={D} bits={bits} page={page} causal={causal} {dt}", flush=True)
    p = Problem(lens, Hkv * G, Hkv, D, bits, page, dt, seed=seed, q_scale=float(np.exp(rng.normal())), spread=0.3,
                spare=(1, WIDE)[seed % 2])
    scale = float(rng.uniform(0.02, 0.3))
    out, lse = p.call(lse=True, causal=causal, scale=scale)
    p.check(out, lse, causal=causal, scale=scale, sample=8)


@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("q_scale,spread", [(30.0, 0.0), (0.0, 0.0), (1.0, 3.0), (8.0, 1.5)])
@pytest.mark.parametrize("G,spare", [(2, 1), (2, WIDE), (3, WIDE), (6, 1), (6, WIDE)])
def test_scores_and_scales_of_all_sizes(D, bits, q_scale, spread, G, spare):
    """Scores that rise by hundreds, none at all, scales that differ by orders of magnitude."""
    print(f"attn q_scale={q_scale} spread={spread} D={D} bits={bits} G={G} spare={spare}", flush=True)
    p = Problem([(1, 700), (2, 64), (1, 333)], 2 * G, 2, D, bits, 64, BF, seed=7, q_scale=q_scale, spread=spread,
                spare=spare)
    out, lse = p.call(lse=True)
    print("share of the tolerance", p.check(out, lse))


def test_scores_that_rise_and_values_that_shrink():
    """The largest value scale comes first, the largest score last, and the other way round."""
    for order in (1, -1):
        p = Problem([(1, 512)], 4, 1, 128, 4, 64, BF, seed=1)
        L = 512
        ramp = np.exp2(-np.arange(L)[::order] / 20.0).astype(np.float32)
        pages = p.table[0, :L // 64]
        vs = p.cache[3].cpu().numpy()
        ks = p.cache[1].cpu().numpy()
        for t in range(L):
            vs[pages[t // 64], 0, t % 64] *= ramp[t]
            ks[pages[t // 64], 0, t % 64] /= ramp[t] ** 0.1
            p.v[0][t] *= np.float64(np.float32(ramp[t]))
        # the products in fp32, as they are stored
        vals = [np.stack([a[pages[t // 64], 0, t % 64] for t in range(L)]) for a in (ks, vs)]
        codes = [np.rint(x / np.abs(x).max(-1, keepdims=True) * 7) for x in (p.k[0], p.v[0])]
        p.k[0], p.v[0] = (c * s[:, None, None].astype(np.float64) for c, s in zip(codes, vals))
        p.ks[0], p.vs_max = vals[0][:, None].astype(np.float64), float(vals[1].max())
        p.cache = (p.cache[0], torch.from_numpy(ks).to(DEV), p.cache[2], torch.from_numpy(vs).to(DEV))
        out, lse = p.call(lse=True)
        p.check(out, lse)


def test_zero_scales():
    """Slots that were cleared: keys and values of zero, not NaN."""
    p = Problem([(1, 100), (1, 64)], 4, 2, 128, 8, 32, FP, seed=2)
    z = tuple(torch.zeros_like(t) for t in p.cache)
    out, lse = w8.attn_kv_cache(p.q.to(DEV), z, torch.tensor(p.table, device=DEV),
                                torch.tensor([100, 64], dtype=torch.int32, device=DEV), lse=True)
    assert not out.any()
    assert np.allclose(_f64(lse), np.log([[100.0], [64.0]]), rtol=8 * U32, atol=0)


def test_strided_queries_scale_and_out():
    p = Problem([(2, 90), (2, 33)], 8, 2, 128, 4, 16, BF, seed=3)
    qkv = torch.randn(4, 12, 128, generator=_gen(1)).to(BF).to(DEV)
    p.q = qkv[:, :8].cpu()
    out = torch.empty(4, 8, 128, dtype=BF, device=DEV)
    got = p.call(ragged=False, q=qkv[:, :8], scale=-0.2, out=out)
    assert got is out
    p.check(out, scale=-0.2)


@pytest.mark.parametrize("pages", [0, 2, 300])
def test_entries_and_lengths_that_contradict_the_sizes(pages):
    """Other sequences are as they would be, and nothing else is written."""
    lens = [(1, 100), (1, 50), (1, 40), (1, 64)]
    p = Problem(lens, 4, 2, 128, 4, 32, BF, seed=4, behind=1, spare=pages)
    table = torch.tensor(p.table, device=DEV)
    table[0, 1], table[0, 2] = 1 << 30, -(1 << 31)
    kv = torch.tensor([100, 2 ** 31 - 1, -2 ** 31, 64], dtype=torch.int32, device=DEV)
    out = torch.full((5, 4, 128), 7.5, dtype=BF, device=DEV)
    p.call(table=table, lens=kv, out=out)
    p.check(out, only=[3])
    assert not out[2].any() and (out[4] == 7.5).all()
    starts = torch.tensor([3, 1, 3, 2 ** 31 - 1, -5], dtype=torch.int32, device=DEV)
    p.call(q_starts=starts, max_q=2, out=out)


@pytest.mark.parametrize("spare", [1, WIDE])
def test_deterministic(spare):
    p = Problem([(1, 3000), (1, 700), (3, 1200)], 8, 4, 128, 4, 64, BF, seed=5, spare=spare)
    a = p.call(lse=True)
    for _ in range(3):
        assert _same(a, p.call(lse=True))


@pytest.mark.parametrize("spare", [1, WIDE])
def test_streams_workspace_and_capture(spare):
    """A captured call replayed over new contents, on another stream, with a workspace of its own."""
    p = Problem([(1, 400), (1, 1300)], 8, 2, 128, 4, 64, BF, seed=6, spare=spare)
    q = p.q.to(DEV)
    ws = torch.empty(w8.attn_workspace_bytes(1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    ws.random_()
    table = torch.tensor(p.table, device=DEV)
    lens = torch.tensor([400, 1300], dtype=torch.int32, device=DEV)
    eager = w8.attn_kv_cache(q, p.cache, table, lens, lse=True)
    out = torch.empty_like(eager[0]), torch.empty_like(eager[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w8.attn_kv_cache(q, p.cache, table, lens, lse=True, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert _same(eager, out)
    # one step: two tokens' rows are written, then attended to
    kn = torch.randn(2, 2, 128, generator=_gen(9)).to(BF).to(DEV)
    vn = torch.randn(2, 2, 128, generator=_gen(10)).to(BF).to(DEV)
    slots = torch.tensor([int(p.table[0, 6]) * 64 + 15, int(p.table[1, 20]) * 64 + 19], dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w8.quant_kv_cache(kn, vn, slots, p.cache)
        got = w8.attn_kv_cache(q, p.cache, table, lens, lse=True)
    for i in range(3):
        kn.copy_(torch.randn(2, 2, 128, generator=_gen(20 + i)))
        vn.copy_(torch.randn(2, 2, 128, generator=_gen(30 + i)))
        lens.copy_(torch.tensor([400 - i, 1300 - 7 * i]))
        graph.replay()
        torch.cuda.synchronize()
        first = tuple(t.clone() for t in got)
        w8.quant_kv_cache(kn, vn, slots, p.cache)
        assert _same(first, w8.attn_kv_cache(q, p.cache, table, lens, lse=True))


def test_empty_batches_and_refusals():
    c = w8.kv_cache_empty(3, 2, 16, 128)
    q = torch.zeros(4, 8, 128, dtype=BF, device=DEV)
    t = torch.zeros(4, 3, dtype=torch.int32, device=DEV)
    n = torch.zeros(4, dtype=torch.int32, device=DEV)
    s = torch.zeros(5, dtype=torch.int32, device=DEV)
    assert w8.attn_kv_cache(q[:0], c, t[:0], n[:0]).shape == (0, 8, 128)
    assert not w8.attn_kv_cache(q, c, t[:, :0], n + 5).any()           # no pages: nothing to see
    for bad in [lambda: w8.attn_kv_cache(q[:3], c, t, n), lambda: w8.attn_kv_cache(q[:, :7], c, t, n),
                lambda: w8.attn_kv_cache(q.float(), c, t, n), lambda: w8.attn_kv_cache(q[..., :64], c, t, n),
                lambda: w8.attn_kv_cache(q.transpose(0, 1), c, t, n), lambda: w8.attn_kv_cache(q, c, t.long(), n),
                lambda: w8.attn_kv_cache(q, c, t, n[:3]), lambda: w8.attn_kv_cache(q, c, t, n, q_starts=s[:4]),
                lambda: w8.attn_kv_cache(q, c, t, n, max_q=2), lambda: w8.attn_kv_cache(q, c, t, n, scale=math.nan),
                lambda: w8.attn_kv_cache(q, c, t, n, q_starts=s, max_q=-1),
                lambda: w8.attn_kv_cache(q, c, t, n, out=q.to(FP)),
                lambda: w8.attn_kv_cache(q, c, t, n, lse=True, out=(q, q)),
                lambda: w8.attn_kv_cache(q, c, t, n, workspace=torch.empty(1024, dtype=torch.uint8, device=DEV)),
                lambda: w8.attn_kv_cache(q, c, t.cpu(), n)]:
        with pytest.raises(w8.W8Error):
            bad()


def test_a_decode_step():
    """Cache write, attention, and the read back of what was attended to, several steps in a row."""
    B, Hq, H, D, page, bits = 3, 8, 2, 128, 16, 4
    c = w8.kv_cache_empty(12, H, page, D, bits=bits)
    table = torch.randperm(12, generator=_gen(0)).to(torch.int32).view(B, 4).to(DEV)
    k = [np.zeros((0, H, D)) for _ in range(B)]
    v = [np.zeros((0, H, D)) for _ in range(B)]
    sc = [np.zeros((0, H)) for _ in range(B)]
    at = 0
    for n in (30, 1, 1, 5, 1):                            # a prompt, answers, drafted tokens
        qkv = torch.randn(B * n, (Hq + 2 * H), D, generator=_gen(n + at)).to(BF)
        g = qkv.to(DEV)
        pos = torch.arange(at, at + n, device=DEV)
        slots = (table[:, pos // page] * page + pos % page).view(-1).to(torch.int32).contiguous()
        w8.quant_kv_cache(g[:, Hq:Hq + H], g[:, Hq + H:], slots, c)
        at += n
        out = w8.attn_kv_cache(g[:, :Hq], c, table, torch.full((B,), at, dtype=torch.int32, device=DEV))
        p = Problem([(n, 0)] * B, Hq, H, D, bits, page, BF, spare=1)
        p.lens, p.q = [(n, at)] * B, qkv[:, :Hq]
        p.vs_max = 0.0
        for b in range(B):
            for x, lo in ((k, Hq), (v, Hq + H)):
                q, s = oc.quant_rows(_np(qkv[b * n:b * n + n, lo:lo + H]), bits)
                x[b] = np.concatenate([x[b], q * s[..., None].astype(np.float64)])
                p.vs_max = max(p.vs_max, float(np.abs(x[b]).max()))
                if x is k:
                    sc[b] = np.concatenate([sc[b], s.astype(np.float64)])
        p.k, p.ks, p.v = k, sc, v
        p.check(out)
    kr, vr = w8.dequant_kv_cache(c, (table[1].repeat_interleave(page) * page
                                     + torch.arange(64, device=DEV) % page)[:at].to(torch.int32), dtype=torch.float32)
    assert np.array_equal(_f64(kr).astype(np.float32), k[1].astype(np.float32))
    assert np.array_equal(_f64(vr).astype(np.float32), v[1].astype(np.float32))
