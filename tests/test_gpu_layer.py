"""GPU parity of the layer around the products: norm_residual_quant,
moe_route_topk and moe_w8a8_block against the 64-bit oracle (oracle/layer.py).

Tolerances, each derived before the first run:
  norm   h and z are rounded once to the 16-bit type (half a step, eps / 2 of
         the value, or half the smallest subnormal) after an fp32 evaluation.
         A sum of K squares, at most 32 per thread in a row, then 6 + 16
         additions, rounds at most 56 times, so the root of the mean is off by
         30 half steps at most, and the products, division and additions
         around it by at most 10 more: 40 * 2^-24 of the norm's term, and
         2^-24 of the sum with the residual.  Codes and scales are the
         oracle's quantiser of the z that was written, bit for bit.
  route  ids equal; weights fp32 roundings (2^-24) of a 64-bit value.
  moe    moe_block's second result (the fp32 steps and the codes they may
         move), and the rounding of the output (2^-24, or 2^-8 in bf16).
"""

import numpy as np
import pytest
import torch

import synth
import w8a8_int8_quantized_amd as w8
from oracle import layer, quant

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = layer.U32


def _np(t):
    return t.detach().float().cpu().numpy() if t.dtype == torch.bfloat16 else t.detach().cpu().numpy()


def _bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def _same(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# -------------------------------------------------------------------- norm
def _norm_inputs(M, K, dt, seed, residual=True, post=True, gate="token"):
    g = _gen(seed)
    def r(*s):
        return torch.randn(*s, generator=g)
    d = {"y": synth.activations(M, K, seed=seed, dtype=dt), "pre_weight": (1 + 0.3 * r(K)).to(dt)}
    if residual:
        d["residual"] = (2 * r(M, K)).to(dt)
    if post:
        d["post_weight"] = (1 + 0.3 * r(K)).to(dt)
    if gate != "none":
        d["gate"] = torch.sigmoid(r(K) if gate == "channel" else r(M, K)).to(dt)
    return d


def _check_norm(d, scale, eps, scheme, got, dt):
    half = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    f = {k: _np(v).astype(np.float64) for k, v in d.items()}
    h, q, s, z = (_np(t) for t in got)
    with np.errstate(all="ignore"):
        h64, t64 = layer.norm_h(f["y"], f.get("residual"), f.get("post_weight"), f.get("gate"), scale, eps)
        e = 40 * U32 * np.abs(t64) + U32 * np.abs(h64)
        bound = half * (np.abs(h64) + e) + e + tiny
        assert (np.abs(h - h64) <= bound).all(), np.max(np.abs(h - h64) / bound)
        z64 = layer.rms_norm(h, f["pre_weight"], eps)
        e = 40 * U32 * np.abs(z64)
        bound = half * (np.abs(z64) + e) + e + tiny
        assert (np.abs(z - z64) <= bound).all(), np.max(np.abs(z - z64) / bound)
    zo = got[3].cpu().numpy() if dt == torch.float16 else synth.to_numpy(got[3])
    rq, rs = quant.quant_act_group(zo) if scheme == w8.W8_SCHEME_BLOCK else quant.quant_act_token(zo)
    assert np.array_equal(q, rq)
    assert np.array_equal(s.view(np.uint32), rs.view(np.uint32))


@pytest.mark.parametrize("scheme", [w8.W8_SCHEME_BLOCK, w8.W8_SCHEME_CHANNEL])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,K", [(1, 128), (3, 256), (2, 1920), (5, 2048), (7, 2176), (2, 7168), (3, 8192), (2, 8320),
                                 (1, 18432), (2, 32768), (333, 384)])
def test_norm(M, K, dt, scheme):
    print(f"norm M={M} K={K} {dt} scheme={scheme}", flush=True)
    d = _norm_inputs(M, K, dt, seed=M + K)
    g = {k: v.to(DEV) for k, v in d.items()}
    got = w8.norm_residual_quant(**g, residual_scale=0.37, eps=1e-5, scheme=scheme, normed=True)
    _check_norm(d, 0.37, 1e-5, scheme, got, dt)
    # without z, and z without codes: the same bits
    assert _same(w8.norm_residual_quant(**g, residual_scale=0.37, eps=1e-5, scheme=scheme), got[:3])
    assert _same(w8.norm_residual_quant(**g, residual_scale=0.37, eps=1e-5, scheme=None, normed=True),
                 (got[0], got[3]))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm_parts(residual, post, gate):
    """Every combination of the optional parts."""
    d = _norm_inputs(9, 640, torch.bfloat16, seed=5, residual=residual, post=post, gate=gate)
    got = w8.norm_residual_quant(**{k: v.to(DEV) for k, v in d.items()}, normed=True)
    _check_norm(d, 1.0, 1e-6, w8.W8_SCHEME_BLOCK, got, torch.bfloat16)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_norm_extreme_rows(dt):
    """Rows of zeros, of subnormals and of large values, a residual that
    cancels the block's output, one large element."""
    d = _norm_inputs(8, 512, dt, seed=6, post=False, gate="none")
    d["y"][0] = 0
    d["residual"][0] = 0
    d["y"][1] = torch.finfo(dt).smallest_normal / 4
    d["residual"][1] = 0
    d["y"][2] = 200.0
    d["residual"][2] = -200.0
    d["y"][3] = 0
    d["residual"][3] = 0
    d["y"][3, 77] = 3e4
    d["y"][4] = torch.linspace(-3e4, 3e4, 512).to(dt)
    got = w8.norm_residual_quant(**{k: v.to(DEV) for k, v in d.items()}, eps=1e-6, normed=True)
    _check_norm(d, 1.0, 1e-6, w8.W8_SCHEME_BLOCK, got, dt)
    assert not got[1][0].any() and not got[1][2].any()


@pytest.mark.parametrize("M,K", [(37, 1152), (260, 18432)])
def test_norm_in_place_and_out(M, K):
    """h into the residual's and into y's own memory; rows behind the last one stay."""
    d = {k: v.to(DEV) for k, v in _norm_inputs(M, K, torch.bfloat16, seed=7).items()}
    want = w8.norm_residual_quant(**d, normed=True)
    for name in ("residual", "y"):
        g = dict(d)
        g[name] = d[name].clone()
        bufs = [torch.full((M + 1, K), 9, dtype=torch.int8, device=DEV),
                torch.full((M + 1, K // 128), 9.0, device=DEV),
                torch.full((M + 1, K), 9.0, dtype=torch.bfloat16, device=DEV)]
        got = w8.norm_residual_quant(**g, normed=True, out=(g[name], *(b[:M] for b in bufs)))
        assert got[0].data_ptr() == g[name].data_ptr() and _same(got, want)
        assert all(bool((b[M] == 9).all()) for b in bufs)


def test_norm_more_rows_than_a_launch_takes():
    """2^20 + 3 rows: two launches, the second of three rows."""
    M, K = (1 << 20) + 3, 128
    y = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    w = torch.ones(K, device=DEV, dtype=torch.bfloat16)
    g = torch.randn(M, K, device=DEV).to(torch.bfloat16)
    got = w8.norm_residual_quant(y, w, residual=y, gate=g, normed=True)
    for part in (slice(0, 5), slice((1 << 20) - 3, M)):
        assert _same(w8.norm_residual_quant(y[part], w, residual=y[part], gate=g[part], normed=True),
                     [t[part] for t in got])


def test_norm_refusals():
    d = {k: v.to(DEV) for k, v in _norm_inputs(4, 256, torch.bfloat16, seed=8).items()}
    bad = [dict(residual=d["residual"][:3]), dict(residual=d["residual"].half()), dict(gate=d["gate"][:2]),
           dict(pre_weight=d["pre_weight"][:128]), dict(post_weight=d["post_weight"].float()),
           dict(y=d["y"].t()), dict(y=d["y"].float()), dict(y=d["y"][:, :192].contiguous()),
           dict(residual=d["residual"].cpu()), dict(scheme=5), dict(scheme=None), dict(out=(d["y"],)), dict(eps=0.0)]
    for b in bad:
        with pytest.raises(w8.W8Error):
            w8.norm_residual_quant(**{**d, **b})
    got = w8.norm_residual_quant(d["y"][:0], d["pre_weight"])
    assert got[0].shape == (0, 256) and got[2].shape == (0, 2)


# ------------------------------------------------------------------ router
def _check_route(logits, got, topk, **kw):
    f = logits.float().numpy()
    bias = kw.get("bias")
    ids, w = layer.route_topk(f, topk, **{**kw, "bias": None if bias is None else bias.numpy()})
    gi, gw = _np(got[0]), _np(got[1]).astype(np.float64)
    assert np.array_equal(gi, ids)
    assert (np.abs(gw - w) <= U32 * 1.001 * np.abs(w) + 1e-45).all(), np.abs(gw - w).max()


def _route(logits, topk, sigmoid=False, bias=None, **kw):
    return w8.moe_route_topk(logits.to(DEV), topk, bias=None if bias is None else bias.to(DEV),
                             score=w8.W8_ROUTE_SIGMOID if sigmoid else w8.W8_ROUTE_SOFTMAX, **kw)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,topk,n_group,topk_group", [
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 8, 2, 1, 1), (9, 61, 6, 1, 1), (4, 64, 8, 8, 4), (7, 65, 5, 1, 1),
    (17, 128, 8, 4, 2), (3, 160, 6, 8, 3), (33, 256, 8, 8, 4), (2, 300, 60, 1, 1), (2, 512, 10, 16, 3),
    (3, 1024, 64, 1, 1), (2, 1023, 7, 1, 1), (2, 1024, 3, 64, 5), (3, 63, 2, 63, 9), (4, 96, 5, 32, 7), (3, 40, 4, 20, 3), (6, 12, 12, 4, 4)])
def test_route(T, E, topk, n_group, topk_group, dt):
    g = _gen(T + E)
    logits = (2 * torch.randn(T, E, generator=g)).to(dt)
    bias = 0.1 * torch.randn(E, generator=g)
    for sigmoid in (False, True):
        for b in (None, bias):
            for top in (1, 2):
                kw = dict(sigmoid=sigmoid, bias=b, n_group=n_group, topk_group=topk_group, group_top=top,
                          renormalise=top == 2, scale=1.0 if top == 1 else 2.5)
                _check_route(logits, _route(logits, topk, **kw), topk, **kw)


def test_route_ties_masks_and_extremes():
    """All logits equal, pairs of equal ones, saturated scores, masked experts
    down to none left, NaN, +inf and the lowest finite value."""
    E = 24
    l = torch.randn(12, E, generator=_gen(3))
    l[0] = 0.5
    l[1] = torch.arange(E).div(4, rounding_mode="floor").float()
    l[2] = 60 + torch.arange(E).float()
    l[3] = -float("inf")
    l[4, 5:] = -float("inf")
    l[5, :20] = float("nan")
    l[6] = float("nan")
    l[7, 3] = float("inf")
    l[7, 9] = float("inf")
    l[8] = torch.finfo(torch.float32).min
    l[9, ::2] = torch.finfo(torch.float32).min
    l[10] = torch.linspace(-1000, 1000, E)
    l[11, 1:] = -float("inf")
    bias = torch.full((E,), -2.0)
    for sigmoid in (False, True):
        for n_group, topk_group in ((1, 1), (6, 3), (24, 9), (2, 1)):
            for b in (None, bias):
                kw = dict(sigmoid=sigmoid, bias=b, n_group=n_group, topk_group=topk_group)
                got = _route(l, 7, **kw)
                _check_route(l, got, 7, **kw)
                assert (got[0][3] == -1).all() and (got[0][6] == -1).all() and not got[1][3].any()
    # a NaN or infinite bias masks or wins, and every slot is written
    bias[4], bias[5], bias[6] = float("nan"), float("inf"), -float("inf")
    out = (torch.full((12, 7), -9, dtype=torch.int32, device=DEV), torch.full((12, 7), -9.0, device=DEV))
    ids, w = _route(l, 7, bias=bias, out=out)
    assert bool(((ids >= -1) & (ids < E)).all()) and bool((w >= 0).all())
    assert not bool(((ids == 4) | (ids == 6)).any())


def test_route_large_batch_and_rows_behind():
    logits = torch.randn(4099, 256, generator=_gen(11))
    ids = torch.full((4100, 8), -7, dtype=torch.int32, device=DEV)
    w = torch.full((4100, 8), -7.0, device=DEV)
    kw = dict(sigmoid=True, n_group=8, topk_group=4, scale=2.5)
    got = _route(logits, 8, out=(ids[:4099], w[:4099]), **kw)
    _check_route(logits, got, 8, **kw)
    assert bool((ids[4099] == -7).all()) and bool((w[4099] == -7).all())


def test_route_refusals():
    l = torch.zeros(4, 16, device=DEV)
    for kw in (dict(topk=0), dict(topk=17), dict(topk=2, n_group=3), dict(topk=9, n_group=4, topk_group=2),
               dict(topk=2, group_top=3), dict(topk=2, score=9), dict(topk=2, bias=torch.zeros(15, device=DEV)),
               dict(topk=2, bias=torch.zeros(16)), dict(topk=2, scale=float("inf"))):
        with pytest.raises(w8.W8Error):
            w8.moe_route_topk(l, **kw)
    with pytest.raises(w8.W8Error):
        w8.moe_route_topk(l.double(), 2)
    with pytest.raises(w8.W8Error):
        w8.moe_route_topk(torch.zeros(16, 4, device=DEV).t(), 2)
    assert w8.moe_route_topk(l[:0], 2)[0].shape == (0, 2)


# ----------------------------------------------------------------- experts
def _moe_inputs(T, topk, E, I, K, seed, ids=None):
    rng = np.random.default_rng(seed)
    x = synth.to_numpy(synth.activations(T, K, seed=seed))
    A, sa = quant.quant_act_group(x)
    def w(*shape):
        return np.clip(np.rint(rng.standard_normal(shape) * 36), -127, 127).astype(np.int8)
    def s(*shape):
        return rng.uniform(0.75, 1.25, shape).astype(np.float32) * np.float32(0.02 / 36)
    if ids is None:
        ids = np.stack([rng.permutation(E)[:topk] if topk <= E else rng.integers(0, E, topk) for _ in range(T)])
    wt = rng.uniform(0.05, 1.0, (T, topk)).astype(np.float32)
    return (A, sa, np.asarray(ids).astype(np.int32).reshape(T, topk), wt, w(E, 2 * I, K), s(E, 2 * I // 128, K // 128),
            w(E, K, I), s(E, K // 128, I // 128))


def _check_moe(args, got32, gotb):
    y, tol = layer.moe_block(*args)
    g = _np(got32).astype(np.float64)
    bound = tol * (1 + U32) + U32 * np.abs(y) + 1e-30
    assert (np.abs(g - y) <= bound).all(), (np.max(np.abs(g - y) / bound), np.linalg.norm(g - y) / np.linalg.norm(y))
    # the bf16 output is the rounding of the same fp32 sums
    assert torch.equal(gotb, got32.to(torch.bfloat16))
    rel = np.linalg.norm(g - y) / max(np.linalg.norm(y), 1e-30)
    assert rel < 1e-2, rel                        # the bound above is not vacuous


def _to(args):
    return [torch.from_numpy(a).to(DEV) for a in args]


@pytest.mark.parametrize("T,topk,E,I,K", [
    (1, 1, 1, 128, 128), (1, 2, 4, 256, 384), (1, 8, 16, 128, 1024), (2, 3, 5, 384, 256), (3, 16, 20, 128, 128),
    (5, 2, 3, 640, 256), (7, 6, 8, 256, 640), (16, 2, 4, 128, 256), (17, 4, 4, 256, 128), (20, 1, 1, 128, 256),
    (32, 3, 6, 128, 384), (33, 2, 2, 256, 256), (48, 1, 1, 384, 128), (64, 8, 12, 128, 256), (64, 1, 1, 256, 128),
    (64, 16, 40, 128, 128), (40, 5, 24, 384, 1280), (64, 2, 3, 1024, 384), (33, 8, 64, 128, 2176), (2, 2, 2, 128, 32768),
    (2, 2, 2, 32768, 128), (64, 1, 1, 128, 32768), (64, 2, 2, 1024, 4096), (40, 4, 5, 512, 384), (1, 1, 300, 128, 128), (4, 2, 8, 1152, 128), (3, 1, 2, 128, 2176)])
def test_moe(T, topk, E, I, K):
    print(f"moe T={T} topk={topk} E={E} I={I} K={K}", flush=True)
    args = _moe_inputs(T, topk, E, I, K, seed=T + E + I)
    t = _to(args)
    got = w8.moe_w8a8_block(*t, out_dtype=torch.float32)
    gotb = w8.moe_w8a8_block(*t)
    torch.cuda.synchronize()
    _check_moe(args, got, gotb)


def test_moe_empty_slots_and_repeats():
    """Ids without an expert (their weights NaN, never read), tokens without
    any, a token that names one expert in every slot, an expert whose rows
    pass 16, 32 and 64, all in one call."""
    T, topk, E, I, K = 64, 8, 10, 256, 256
    rng = np.random.default_rng(1)
    ids = rng.integers(0, E, (T, topk))
    ids[rng.random((T, topk)) < 0.3] = -1
    ids[5] = -1
    ids[6] = [E, E + 1, -2, 2**31 - 1, -2**31, E, -1, 4096]
    ids[7] = 3
    ids[8:40, 0] = 9
    ids[8:24, 1] = 9
    ids[0:18] = np.where(ids[0:18] == 2, 1, ids[0:18])
    args = _moe_inputs(T, topk, E, I, K, seed=2, ids=ids)
    args[3][(ids < 0) | (ids >= E)] = np.nan
    t = _to(args)
    ws = torch.full((w8.moe_workspace_bytes(T, topk, I, K),), 0xFF, dtype=torch.uint8, device=DEV)
    buf = torch.full((T + 1, K), 5.0, device=DEV)
    got = w8.moe_w8a8_block(*t, out=buf[:T], workspace=ws)
    _check_moe(args, got, w8.moe_w8a8_block(*t))
    assert not got[5].any() and not got[6].any() and bool((buf[T] == 5).all())
    again = w8.moe_w8a8_block(*t, out_dtype=torch.float32)
    assert torch.equal(again.view(torch.int32), got.view(torch.int32))


@pytest.mark.parametrize("T,topk", [(64, 16), (12, 16), (30, 8)])
def test_moe_one_expert_takes_all(T, topk):
    """Every slot of every token names the same expert: its rows pass the
    tokens and take several passes."""
    args = _moe_inputs(T, topk, 3, 128, 256, seed=9, ids=np.full((T, topk), 1))
    t = _to(args)
    _check_moe(args, w8.moe_w8a8_block(*t, out_dtype=torch.float32), w8.moe_w8a8_block(*t))


def test_moe_weights_beyond_four_gigabytes():
    """160 experts of K = 7168, I = 2048 (4.7 GB of W_gate_up): the last ones
    against the oracle on their own weights."""
    T, topk, E, I, K = 2, 2, 160, 2048, 7168
    used = [3, 158, 159]
    small = _moe_inputs(T, topk, len(used), I, K, seed=8, ids=[[2, 0], [1, 2]])
    A, sa, ids, wt, w13, s13, w2, s2 = _to(small)
    big = []
    for v in (w13, s13, w2, s2):
        full = torch.ones(E, *v.shape[1:], dtype=v.dtype, device=DEV)
        full[used] = v
        big.append(full)
    at = torch.tensor(used, dtype=torch.int32, device=DEV)[ids.long()]
    got = w8.moe_w8a8_block(A, sa, at, wt, *big, out_dtype=torch.float32)
    _check_moe(small, got, w8.moe_w8a8_block(A, sa, at, wt, *big))


def test_moe_none_chosen():
    args = _moe_inputs(3, 2, 4, 128, 128, seed=4, ids=np.full((3, 2), -1))
    assert not w8.moe_w8a8_block(*_to(args)).any()


def test_moe_refusals():
    t = _to(_moe_inputs(4, 2, 4, 128, 256, seed=5))
    names = ["A", "a_scale", "topk_ids", "topk_weights", "W_gate_up", "gate_up_scale", "W_down", "down_scale"]
    for i, bad in [(0, t[0].float()), (0, t[0].cpu()), (1, t[1][:, :1].contiguous()), (2, t[2].long()),
                   (3, t[3][:3]), (4, t[4][:, :, :128].contiguous()), (5, t[5].half()), (6, t[6].transpose(1, 2)),
                   (7, t[7][:3])]:
        with pytest.raises(w8.W8Error):
            w8.moe_w8a8_block(*[bad if k == i else v for k, v in enumerate(t)])
    with pytest.raises(w8.W8Error):
        w8.moe_w8a8_block(*t, out_dtype=torch.float16)
    with pytest.raises(w8.W8Error, match="workspace"):
        w8.moe_w8a8_block(*t, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    big = _to(_moe_inputs(65, 1, 2, 128, 128, seed=6))
    with pytest.raises(w8.W8Error):
        w8.moe_w8a8_block(*big)
    assert w8.moe_w8a8_block(*[v[:0] if k < 4 else v for k, v in enumerate(t)]).shape == (0, 256)
    assert len(names) == len(t)


# ------------------------------------------------------------ all together
def _step(x, r, p, ws, out=None):
    """The feed-forward half of a layer: norm, router, experts, norm behind
    them with the residual, and the next layer's codes."""
    h, q, s, z = w8.norm_residual_quant(x, p["w0"], residual=r, normed=True)
    logits = torch.mm(z.float(), p["router"])
    ids, wt = w8.moe_route_topk(logits, 4, bias=p["bias"], score=w8.W8_ROUTE_SIGMOID, n_group=4, topk_group=2,
                                scale=2.5)
    y = w8.moe_w8a8_block(q, s, ids, wt, p["w13"], p["s13"], p["w2"], p["s2"], workspace=ws)
    h2, q2, s2 = w8.norm_residual_quant(y, p["w1"], residual=h, post_weight=p["w2n"], residual_scale=0.5)
    return dict(h=h, q=q, s=s, z=z, logits=logits, ids=ids, wt=wt, y=y, h2=h2, q2=q2, s2=s2)


def _step_params(K, I, E, seed):
    g = _gen(seed)
    args = _moe_inputs(1, 4, E, I, K, seed)
    p = {"w0": 1 + 0.2 * torch.randn(K, generator=g), "w1": 1 + 0.2 * torch.randn(K, generator=g),
         "w2n": 1 + 0.2 * torch.randn(K, generator=g)}
    p = {k: v.to(torch.bfloat16) for k, v in p.items()}
    p.update(router=torch.randn(K, E, generator=g) / K ** 0.5, bias=0.05 * torch.randn(E, generator=g),
             w13=torch.from_numpy(args[4]), s13=torch.from_numpy(args[5]), w2=torch.from_numpy(args[6]),
             s2=torch.from_numpy(args[7]))
    return p, {k: v.to(DEV) for k, v in p.items()}


@pytest.mark.parametrize("T", [1, 19, 64])
def test_feed_forward_half_of_a_layer(T):
    """Each step of the run against the oracle on what the step before wrote."""
    K, I, E = 512, 256, 16
    cpu, p = _step_params(K, I, E, seed=20)
    x, r = synth.activations(T, K, seed=21), synth.activations(T, K, seed=22)
    o = _step(x.to(DEV), r.to(DEV), p, None)
    _check_norm({"y": x, "residual": r, "pre_weight": cpu["w0"]}, 1.0, 1e-6, w8.W8_SCHEME_BLOCK,
                (o["h"], o["q"], o["s"], o["z"]), torch.bfloat16)
    _check_route(o["logits"].cpu(), (o["ids"], o["wt"]), 4, bias=cpu["bias"], sigmoid=True, n_group=4, topk_group=2,
                 scale=2.5)
    args = [_np(o[k]) for k in ("q", "s", "ids", "wt")] + [cpu[k].numpy() for k in ("w13", "s13", "w2", "s2")]
    y, tol = layer.moe_block(*args)
    assert (np.abs(_np(o["y"]) - y) <= tol + 2.0 ** -8 * (np.abs(y) + tol)).all()
    h2, q2, s2, z2 = w8.norm_residual_quant(o["y"], p["w1"], residual=o["h"], post_weight=p["w2n"],
                                            residual_scale=0.5, normed=True)
    assert _same((h2, q2, s2), (o["h2"], o["q2"], o["s2"]))
    _check_norm({"y": o["y"].cpu(), "residual": o["h"].cpu(), "pre_weight": cpu["w1"], "post_weight": cpu["w2n"]},
                0.5, 1e-6, w8.W8_SCHEME_BLOCK, (h2, q2, s2, z2), torch.bfloat16)


def test_layer_graph_replays_and_streams():
    """The run captured into a graph and replayed with changed inputs, eager
    work between the replays; and two streams at once with a workspace each."""
    K, I, E, T = 512, 256, 16, 24
    _, p = _step_params(K, I, E, seed=30)
    ws = torch.empty(w8.moe_workspace_bytes(T, 4, I, K), dtype=torch.uint8, device=DEV)
    xs = [synth.activations(T, K, seed=40 + i).to(DEV) for i in range(4)]
    r = synth.activations(T, K, seed=50).to(DEV)
    want = [_step(x, r, p, None) for x in xs]
    x = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(x, r, p, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _step(x, r, p, ws)
    for i in (0, 1, 2, 3, 1, 0):
        x.copy_(xs[i])
        graph.replay()
        eager = _step(xs[(i + 1) % 4], r, p, None)
        torch.cuda.synchronize()
        assert all(_same((got[k],), (want[i][k],)) for k in want[i]), i
        assert all(_same((eager[k],), (want[(i + 1) % 4][k],)) for k in eager), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    torch.cuda.synchronize()
    for k in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(_step(xs[(k + i) % 4], r, p, None))
    torch.cuda.synchronize()
    for i in range(2):
        for k in range(6):
            w = want[(k + i) % 4]
            assert all(_same((outs[i][k][n],), (w[n],)) for n in w)


# ----------------------------------------------------------- drawn shapes
@pytest.mark.parametrize("seed", range(24))
def test_moe_drawn(seed):
    """Tokens, slots, experts and sides drawn over the small end of their
    ranges; skewed ids (some experts take most rows), a share of them empty."""
    rng = np.random.default_rng(1000 + seed)
    T, topk, E = int(rng.integers(1, 65)), int(rng.integers(1, 17)), int(2 ** rng.uniform(0, 8))
    I, K = 128 * int(rng.integers(1, 6)), 128 * int(rng.integers(1, 6))
    if E * I * K > 1 << 24:
        E = max(1, (1 << 24) // (I * K))
    p = rng.random(E) ** 3 + 1e-3
    ids = rng.choice(E, size=(T, topk), p=p / p.sum())
    ids[rng.random((T, topk)) < rng.choice([0.0, 0.2, 0.9])] = -1
    print(f"moe T={T} topk={topk} E={E} I={I} K={K}", flush=True)
    args = _moe_inputs(T, topk, E, I, K, seed=seed, ids=ids)
    args[3][ids < 0] = np.nan
    t = _to(args)
    got = w8.moe_w8a8_block(*t, out_dtype=torch.float32)
    _check_moe(args, got, w8.moe_w8a8_block(*t))
    empty = (ids < 0).all(1)
    assert not got[torch.from_numpy(empty).to(DEV)].any()


@pytest.mark.parametrize("seed", range(16))
def test_norm_drawn(seed):
    rng = np.random.default_rng(2000 + seed)
    M, K = int(2 ** rng.uniform(0, 9.5)), 128 * int(2 ** rng.uniform(0, 7.2))
    dt = [torch.bfloat16, torch.float16][int(rng.integers(2))]
    d = _norm_inputs(M, K, dt, seed=seed, residual=bool(rng.integers(2)), post=bool(rng.integers(2)),
                     gate=["none", "channel", "token"][int(rng.integers(3))])
    scale, scheme = float(rng.uniform(-1, 2)), [w8.W8_SCHEME_BLOCK, w8.W8_SCHEME_CHANNEL][int(rng.integers(2))]
    print(f"norm M={M} K={K} {dt} {sorted(d)} scale={scale} scheme={scheme}", flush=True)
    got = w8.norm_residual_quant(**{k: v.to(DEV) for k, v in d.items()}, residual_scale=scale, scheme=scheme,
                                 normed=True)
    _check_norm(d, scale, 1e-6, scheme, got, dt)


@pytest.mark.parametrize("seed", range(16))
def test_route_drawn(seed):
    rng = np.random.default_rng(3000 + seed)
    groups = int(rng.choice([1, 1, 2, 5, 16]))
    E, T = groups * int(2 ** rng.uniform(0, 10 - np.log2(groups))), int(2 ** rng.uniform(0, 6))
    kept = int(rng.integers(1, groups + 1))
    topk = int(rng.integers(1, min(64, kept * (E // groups)) + 1))
    l = torch.from_numpy(rng.standard_normal((T, E)) * 2).to([torch.float32, torch.bfloat16][int(rng.integers(2))])
    l[torch.from_numpy(rng.random((T, E)) < rng.choice([0.0, 0.3, 0.95]))] = -float("inf")
    bias = torch.from_numpy(rng.standard_normal(E) * 0.3).float() if rng.integers(2) else None
    kw = dict(sigmoid=bool(rng.integers(2)), bias=bias, n_group=groups, topk_group=kept,
              group_top=int(rng.integers(1, 3)), renormalise=bool(rng.integers(2)), scale=float(rng.uniform(0.5, 3)))
    print(f"route T={T} E={E} topk={topk} {kw['n_group']}/{kept}", flush=True)
    _check_route(l, _route(l, topk, **kw), topk, **kw)
