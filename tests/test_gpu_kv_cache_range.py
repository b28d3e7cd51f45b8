"""Attention over the quantised cache where scores and scales are far from 1.

Scores without a rounding.  Codes and queries are small integers but for one
channel, key scales are powers of two, and a call's scale of fp32(ln 2) 2^j is
exactly 2^j where the kernels hold it (in base 2: ln 2 is off by 2.7e-9 of
itself, less than half a step).  All sums of a score stay below 2^24, so the
scores are whole multiples of a power of two without an error, however large,
and the formula in 64 bits on them is what the call has to give but for the
roundings behind the scores.  Tolerances, derived before the first run (u32 =
2^-24):
  terms  exp2 (2 units), the product with the value's scale, fp16 (2^-11); in
         fp16 what lies below the normal range is off by 2^-25, where the
         largest term so far is 2^9 or more: 2^-34 of it.
  sums   as in test_gpu_kv_cache.py: (n / 32 + 40) u32, twice in out.
  out    + the output's rounding.   lse: sums + 4 u32 (|lse| + 1).
"""

import math

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_amd as w8
from oracle import cache as oc
from test_gpu_kv_cache import BF, DEV, FORMS, FP, U32, WIDE, Problem, _empty_np, _f64, _to_gpu

pytestmark = pytest.mark.gpu
LN2 = float(np.float32(math.log(2)))
# query heads to a key head, query tokens: row tiles of 4, 8, 16, 32 and 64
ROWS = [(2, 1), (6, 1), (5, 3), (4, 530), (4, 5100)]


class Exact:
    """Sequences of L tokens; scores in base 2 are f times whole numbers."""

    def __init__(self, lens, n, G, Hkv, D, bits, dt, f, seed, spare=1, page=32, vs_to=10):
        rng = np.random.default_rng(seed)
        top = 7 if bits == 4 else 127
        offset = {(4, FP): 72, (4, BF): 136, (8, FP): 1152, (8, BF): 128}[bits, dt]
        self.Hkv, self.G, self.D, self.dt, self.f, self.n, self.lens = Hkv, G, D, dt, f, n, lens
        e_max = min(15, int(math.log2((1 << 24) / (offset + top) - D - 8)))
        per = [-(-L // page) for L in lens]
        pages = sum(per) + 1
        c = _empty_np(pages, Hkv, page, D, bits, seed)
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(per) + spare), -7, np.int32)
        self.kq, self.vq, self.vs, at = [], [], [], 0
        for b, L in enumerate(lens):
            self.table[b, :per[b]] = order[at:at + per[b]]
            at += per[b]
            kq = rng.integers(-1, 2, (L, Hkv, D))
            kq[..., 0] = top
            vq = rng.integers(-top, top + 1, (L, Hkv, D))
            vs = np.exp2(rng.uniform(-20, vs_to, (L, Hkv))).astype(np.float32)
            for t in range(L):
                for h in range(Hkv):
                    oc.put(c, self.table[b, t // page], t % page, h, kq[t, h], np.float32(0.125), vq[t, h], vs[t, h], bits)
            self.kq.append(kq)
            self.vq.append(vq)
            self.vs.append(vs)
        T, Hq = n * len(lens), Hkv * G
        q = rng.integers(-1, 2, (T, Hq, D))
        # every row has a size of its own: near 0, and of either sign up to the largest
        size = rng.integers(-1, e_max + 1, (T, Hq))
        q[..., 0] = np.where(size < 0, 0, np.exp2(size)) * rng.choice([-1, 1], (T, Hq))
        self.q = q
        assert (np.abs(q).sum(-1) * (offset + top)).max() < 1 << 24
        self.cache = _to_gpu(c, bits)

    def call(self, causal):
        i32 = {"dtype": torch.int32, "device": DEV}
        return w8.attn_kv_cache(torch.from_numpy(self.q).to(self.dt).to(DEV), self.cache, torch.tensor(self.table, **i32),
                                torch.tensor(self.lens, **i32), causal=causal, scale=LN2 * self.f * 8, lse=True)

    def check(self, out, lse, causal, sample):
        half = torch.finfo(self.dt).eps / 2
        tiny = torch.finfo(self.dt).smallest_normal * half
        o, z = _f64(out), _f64(lse)
        rng = np.random.default_rng(1)
        for b, L in enumerate(self.lens):
            for i in sorted({0, self.n - 1} | set(rng.integers(0, self.n, sample).tolist())):
                seen = max(0, L - self.n + i + 1) if causal else L
                for j in range(self.Hkv * self.G):
                    r, h = b * self.n + i, j // self.G
                    if seen == 0:
                        assert not o[r, j].any() and z[r, j] == -math.inf
                        continue
                    s = (self.kq[b][:seen, h] @ self.q[r, j]) * float(self.f)
                    vs = self.vs[b][:seen, h].astype(np.float64)
                    v = self.vq[b][:seen, h] * vs[:, None]
                    p = np.exp2(s - s.max())
                    total = p.sum()
                    want, mag = p @ v / total, p @ np.abs(v) / total
                    sums = (seen / 32 + 40) * U32
                    e = (2.0 ** -11 + 4 * U32 + 2 * sums) * mag + seen * 2.0 ** -34 * 127 * (p * vs).max() / total
                    bound = half * (np.abs(want) + e) + e + tiny
                    d = np.abs(o[r, j] - want)
                    # values go to 127 * 2^10 = 130048, fp16 to 65504: what lies past that within the bound is infinite
                    d[np.isinf(o[r, j]) & (o[r, j] * want > 0) & (np.abs(want) + bound > torch.finfo(self.dt).max)] = 0
                    assert (d <= bound).all(), (b, i, j, s.max(), float((d / bound).max()))
                    lz = math.log(2) * (s.max() + math.log2(total))
                    assert abs(z[r, j] - lz) <= sums + 4 * U32 * (abs(lz) + 1), (b, i, j, z[r, j], lz)


@pytest.mark.parametrize("f", [2.0 ** -2, 2.0, 16.0, 2.0 ** 10, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("spare", [1, WIDE])
def test_scores_of_every_size(D, bits, dt, f, spare):
    """Rows of all sizes side by side, some past any step of fp32 that a softmax could resolve."""
    for G, n in ROWS[:3]:
        print(f"attn far scores D={D} bits={bits} {dt} f={f} G={G} n={n} spare={spare}", flush=True)
        p = Exact([700, 64, 333], n, G, 2, D, bits, dt, f, seed=G, spare=spare)
        p.check(*p.call(True), causal=True, sample=3)


@pytest.mark.parametrize("f", [2.0, 2.0 ** 10, 2.0 ** 100])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("G,n", ROWS[3:])
def test_scores_of_every_size_in_larger_tiles(D, bits, dt, f, G, n):
    print(f"attn far scores D={D} bits={bits} {dt} f={f} G={G} n={n}", flush=True)
    p = Exact([333], n, G, 2, D, bits, dt, f, seed=n)
    p.check(*p.call(False), causal=False, sample=20)


@pytest.mark.parametrize("spare", [1, WIDE])
@pytest.mark.parametrize("scale", [1e5, -1e6, 1e7, -1e9, 1e12, 1e20, 1e30])
def test_scales_far_from_one(scale, spare):
    """Ordinary keys and queries: finite, no larger than the largest value, lse the largest score."""
    for G, dt in ((2, BF), (8, FP), (24, BF)):
        p = Problem([(1, 300), (3, 100), (5, 5)], 2 * G, 2, 128, 4, 32, dt, seed=G, spare=spare)
        out, lse = p.call(scale=scale, lse=True)
        o, z, q = _f64(out), _f64(lse), _f64(p.q)
        for b, (n, L) in enumerate(p.lens):
            for i in range(n):
                for j in range(2 * G):
                    r, h = int(p.starts[b]) + i, j // G
                    seen = L - n + i + 1
                    k, v = p.k[b][:seen, h], p.v[b][:seen, h]
                    s = scale * (k @ q[r, j])
                    # a score is off by the steps that test_gpu_kv_cache.py derives for it
                    off = abs(scale) * float(p.ks[b][:seen, h].max()) * U32 * (
                        6 * math.sqrt(p.D + 1) * (1152 * 2 + 127) * np.abs(q[r, j]).sum()) + 8 * U32 * np.abs(s).max()
                    assert abs(z[r, j] - s.max()) <= off + math.log(seen) + 1, (b, i, j)
                    assert (np.abs(o[r, j]) <= np.abs(v).max(0) * (1 + 2.0 ** -7)).all(), (b, i, j)


def test_a_score_past_the_range():
    """One that overflows counts as infinite: among finite ones it weighs nothing or gives NaN."""
    p = Exact([40], 1, 2, 1, 128, 4, FP, 2.0 ** 100, seed=3)
    p.q[0, :, 1:] = 0
    p.q[0, :, 0] = [0, 16]
    k = p.cache[1].clone()
    at = p.table[0, 0]
    k[at, 0, 7] *= 2.0 ** 24                     # one token's score: 7 * 16 * 2^124, past 2^128
    p.cache = (p.cache[0], k, *p.cache[2:])
    out, lse = p.call(True)
    assert torch.isfinite(out[0, 0]).all() and abs(float(lse[0, 0]) - math.log(40)) < 1e-4
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    p.q[0, :, 0] = [0, -16]
    out, lse = p.call(True)
    keep = np.arange(40) != 7
    want = p.vq[0][keep, 0] * p.vs[0][keep, :].astype(np.float64)
    assert np.allclose(_f64(out)[0, 1], want.mean(0), rtol=0, atol=2.0 ** -9 * np.abs(want).mean(0).max())
    assert abs(float(lse[0, 1]) / (-7 * 16 * 2.0 ** 100 * math.log(2)) - 1) < 4 * U32


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("G,n,spare", [(1, 3, 1), (1, 3, WIDE), (2, 4, 1), (5, 3, WIDE), (3, 40, 1), (4, 530, 1), (4, 5100, 1)])
def test_hidden_tokens_of_any_value(G, n, spare, D, bits, dt, bad):
    """The last tokens' scales are infinite or NaN: queries before them do not see that, and lse never does."""
    print(f"attn hidden values G={G} n={n} spare={spare} D={D} bits={bits} {dt} {bad}", flush=True)
    L = n + 45
    p = Problem([(n, L), (n, n)], 2 * G, 2, D, bits, 32, dt, seed=G + n, spare=spare)
    want, want_lse = p.call(lse=True)
    _, ks, _, vs = p.cache
    for b, kv in enumerate((L, n)):
        for t in (kv - 1, kv - 2):
            at = int(p.table[b, t // 32]), slice(None), t % 32
            vs[at] = bad
            if t == kv - 1:
                ks[at] = bad
    out, lse = p.call(lse=True)
    for b in range(2):
        rows = slice(int(p.starts[b]), int(p.starts[b]) + n)
        o, z, full = _f64(out[rows]), _f64(lse[rows]), _f64(want_lse[rows])
        assert np.isfinite(o[:-2]).all() and not np.isfinite(o[-2:]).all(-1).any()
        assert np.allclose(z[:-1], full[:-1], rtol=0, atol=1e-5 * (1 + np.abs(full).max()))
        # the queries that see none of it: what they gave before, but for references that moved elsewhere
        d = np.abs(o[:-2] - _f64(want[rows])[:-2])
        assert (d <= 2 * torch.finfo(dt).eps * (1 + np.abs(o[:-2]))).all()


@pytest.mark.parametrize("mean", [0.0, 8.0])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
def test_scores_themselves(D, bits, dt, mean):
    """Sequences of one token: lse is the score.  Its tolerance as in test_gpu_kv_cache.py, but with what each form adds
    to its codes (the largest of them there), for queries around 0 and around 8."""
    p = Problem([(1, 1)] * 40, 16, 4, D, bits, 16, dt, seed=D + bits)
    p.q = (p.q.float() + mean).to(dt)
    out, lse = p.call(ragged=False, lse=True)
    z, q = _f64(lse), _f64(p.q)
    offset, top = {(4, FP): 72, (4, BF): 136, (8, FP): 1152, (8, BF): 128}[bits, dt], 7 if bits == 4 else 127
    worst = worst_off = 0.0
    for b in range(40):
        for j in range(16):
            h = j // 4
            s = D ** -0.5 * (p.k[b][0, h] @ q[b, j])
            qa = np.abs(q[b, j]).sum()
            codes = offset * (qa + abs(q[b, j].sum())) + top * qa
            # (and the logarithm of a sum that is one power of two: 4 u32 (|s| + 1))
            bound = 6 * math.sqrt(D + 1) * U32 * codes * D ** -0.5 * p.ks[b][0, h] + U32 * (10 * abs(s) + 8)
            worst, worst_off = max(worst, abs(z[b, j] - s) / bound), max(worst_off, abs(z[b, j] - s))
            assert abs(z[b, j] - s) <= bound, (b, j, s, z[b, j])
    print(f"scores D={D} bits={bits} {dt} mean={mean}: off by {worst_off:.2e} at most, {worst:.3f} of the tolerance")


@pytest.mark.parametrize("f", [0.25, 2.0, 2.0 ** 40])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("G,n,spare", [(2, 1, 1), (6, 1, WIDE), (5, 3, 1), (4, 530, 1), (4, 5100, 1)])
def test_values_of_every_size(G, n, spare, bits, f):
    """Value scales from 2^-20 to 2^99 side by side: probabilities are lost from 2^-36 of the largest on only."""
    p = Exact([333, 64], n, G, 2, 128, bits, BF, f, seed=n, spare=spare, vs_to=99)
    p.check(*p.call(False), causal=False, sample=6)


@pytest.mark.parametrize("L", [1, 10, 40, 700])
@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("G", [2, 6, 12])
@pytest.mark.parametrize("spare", [1, WIDE])
def test_scores_above_the_range_give_nan(G, D, bits, L, spare):
    """In out and in lse, whether one wave holds the sequence or many do; rows beside them are as ever."""
    p = Exact([L], 1, G, 1, D, bits, FP, 2.0 ** 100, seed=L, spare=spare)
    p.q[0, 1, 1:] = 0
    p.q[0, 1, 0] = 16
    t = L // 2
    k = p.cache[1].clone()
    k[p.table[0, t // 32], 0, t % 32] *= 2.0 ** 24     # that token's score: 16 * 7 (or 127) * 2^124
    rest = [j for j in range(G) if j != 1]
    p.q[0, rest] = 0
    p.cache = (p.cache[0], k, *p.cache[2:])
    out, lse = p.call(True)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert torch.isfinite(out[0, rest]).all() and np.allclose(_f64(lse)[0, rest], math.log(L), rtol=0, atol=1e-5)
