"""The quantised cache and the attention over it without a GPU: every call
fails its argument checks or is a no-op, so no kernel launches; and pins of
their oracle by hand-worked values."""

import ctypes

import numpy as np
import pytest

import w8a8_int8_quantized_amd as w8
from oracle import cache, int4, quant

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EVAL = 0, -1, -2, -3, -4, -6, -8
P = ctypes.c_void_p(1 << 20)          # aligned fake address, never dereferenced
P4 = ctypes.c_void_p((1 << 20) + 4)
P2 = ctypes.c_void_p((1 << 20) + 2)
N = ctypes.c_void_p(0)
BF, FP = w8.W8_BF16, w8.W8_FP32


def _write(k=P, v=P, dtype=BF, k_stride=1024, v_stride=1024, slots=P, T=4, H=8, D=128, bits=4, pages=3, page=64, kc=P,
           ks=P, vc=P, vs=P):
    return w8.lib.quant_kv_cache(k, v, dtype, k_stride, v_stride, slots, T, H, D, bits, pages, page, kc, ks, vc, vs, N)


def _read(kc=P, ks=P, vc=P, vs=P, slots=P, T=4, H=8, D=128, bits=4, pages=3, page=64, k=P, v=P, dtype=BF):
    return w8.lib.dequant_kv_cache(kc, ks, vc, vs, slots, T, H, D, bits, pages, page, k, v, dtype, N)


def _attn(q=P, dtype=BF, q_stride=4096, kc=P, ks=P, vc=P, vs=P, table=P, lens=P, starts=P, B=2, T=4, max_q=4, Hq=32,
          H=8, D=128, bits=4, pages=3, page=64, max_pages=2, scale=0.1, causal=1, out=P, lse=P, ws=P, nbytes=1 << 40):
    return w8.lib.attn_kv_cache(q, dtype, q_stride, kc, ks, vc, vs, table, lens, starts, B, T, max_q, Hq, H, D, bits,
                                pages, page, max_pages, scale, causal, out, lse, ws, nbytes, N)


@pytest.mark.parametrize("call", [_write, _read, _attn])
def test_cache_argument_checks(call):
    for bits in (0, 2, 16):
        assert call(bits=bits) == EDTYPE
    for D in (0, 32, 96, 512, -128):
        assert call(D=D) == ESHAPE
    for page in (0, 8, 24, -16, (1 << 20) + 16):
        assert call(page=page) == ESHAPE
    assert call(pages=0) == ESHAPE and call(pages=1 << 31) == ESHAPE and call(pages=1 << 25) == ESHAPE
    assert call(H=0) == ESHAPE and call(H=-8) == ESHAPE and call(H=1 << 13) == ESHAPE
    assert call(dtype=w8.W8_I32) == EDTYPE and call(T=-1) == ESHAPE
    for name in ("kc", "ks", "vc", "vs"):
        assert call(**{name: N}) == ENULL, name
        assert call(**{name: P4}) == EALIGN, name


def test_write_and_read_argument_checks():
    assert _write(dtype=FP) == EDTYPE
    for name in ("k_stride", "v_stride"):
        assert _write(**{name: 1020}) == ESHAPE and _write(**{name: -1024}) == ESHAPE
    assert _write(T=(1 << 24) + 1) == ESHAPE and _read(T=(1 << 24) + 1) == ESHAPE
    for call in (_write, _read):
        for name in ("k", "v", "slots"):
            assert call(**{name: N}) == ENULL, name
            assert call(**{name: P2}) == EALIGN, name
        assert call(k=P4) == EALIGN and call(v=P4) == EALIGN
        assert call(T=0, k=N, v=N, slots=N, kc=N, ks=N, vc=N, vs=N) == OK


def test_attn_argument_checks():
    assert _attn(dtype=FP) == EDTYPE
    assert _attn(Hq=0) == ESHAPE and _attn(Hq=12) == ESHAPE and _attn(Hq=4) == ESHAPE and _attn(Hq=1 << 13) == ESHAPE
    assert _attn(B=-1) == ESHAPE and _attn(max_q=-1) == ESHAPE and _attn(max_q=5) == ESHAPE
    assert _attn(q_stride=4100) == ESHAPE and _attn(q_stride=-4096) == ESHAPE
    assert _attn(starts=N) == ESHAPE                     # 4 tokens are not 2 times 4
    assert _attn(max_pages=-1) == ESHAPE and _attn(max_pages=1 << 26) == ESHAPE
    assert _attn(T=1 << 27) == ESHAPE                    # T * Hq
    # more units of work than 32 bits count
    assert _attn(B=1 << 16, T=1 << 16, max_q=1 << 10, max_pages=1 << 12) == ESHAPE
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert _attn(scale=scale) == EVAL
    for name in ("q", "table", "lens", "out", "ws"):
        assert _attn(**{name: N}) == ENULL, name
    for name in ("q", "out", "ws"):
        assert _attn(**{name: P4}) == EALIGN, name
    for name in ("table", "lens", "starts", "lse"):
        assert _attn(**{name: P2}) == EALIGN, name
    need = w8.lib.attn_workspace_bytes(4, 32, 8, 128)
    assert need > 0 and _attn(nbytes=need - 1) == EWS
    for none in ({"B": 0}, {"T": 0, "max_q": 0}, {"max_q": 0}):
        assert _attn(q=N, out=N, ws=N, nbytes=0, lens=N, table=N, **none) == OK
    for bad in ((-1, 32, 8, 128), (4, 33, 8, 128), (4, 32, 0, 128), (4, 32, 8, 100), (4, 4, 8, 128)):
        assert w8.lib.attn_workspace_bytes(*bad) == ESHAPE


def test_binding_refusals():
    import torch
    for kw in ({"bits": 5}, {"head_dim": 96}, {"page_size": 20}):
        with pytest.raises(w8.W8Error):
            w8.kv_cache_empty(**{"pages": 2, "kv_heads": 2, "page_size": 16, "head_dim": 64, "device": "cpu", **kw})
    c = w8.kv_cache_empty(2, 3, 32, 64, bits=4, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 3, 32, 32), (2, 3, 32), (2, 3, 8, 16, 4, 2), (2, 3, 32)]
    assert [t.dtype for t in w8.kv_cache_empty(2, 3, 32, 256, bits=8, device="cpu")] == [
        torch.int8, torch.float32, torch.int8, torch.float32]
    x = torch.zeros(4, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(w8.W8Error):
        w8.quant_kv_cache(x, x, i, c)                    # tensors on the CPU
    with pytest.raises(w8.W8Error):
        w8.dequant_kv_cache(c, i)
    with pytest.raises(w8.W8Error):
        w8.attn_kv_cache(x, c, i.view(4, 1), i)


# ------------------------------------------------------------------ oracle
def test_oracle_rows_are_the_library_quantisers():
    """A row of 128 channels is a group of the 8-bit and of the 4-bit group quantiser."""
    x = np.random.default_rng(3).normal(size=(9, 128)).astype(np.float16)
    x[4] = 0
    q, s = cache.quant_rows(x, 8)
    rq, rs = quant.quant_act_group(x)
    assert np.array_equal(q, rq) and np.array_equal(s, rs[:, 0])
    q, s = cache.quant_rows(x, 4)
    rq, rs = int4.quant_weight_int4_group(x)
    assert np.array_equal(q, rq) and np.array_equal(s, rs[:, 0])
    assert np.array_equal(cache.row_bytes(q, 4), int4.pack_int4(rq))


def test_oracle_layout_by_hand():
    c = (np.zeros((2, 1, 16, 32), np.uint8), np.zeros((2, 1, 16), np.float32), np.zeros((2, 1, 4, 16, 4, 2), np.uint8),
         np.zeros((2, 1, 16), np.float32))
    q = np.arange(64) % 15 - 7
    cache.put(c, 1, 6, 0, q, 0.5, -q, 0.25, 4)
    assert c[0][1, 0, 6, 0] == 1 + 16 * 2 and c[0][1, 0, 6, 7] == 15 + 16 * 1       # codes -7, -6; 7, -7
    # channels 4, 5 of the value are byte 0 of sixteenth 1, in the second block of four tokens, third place
    assert c[2][1, 0, 1, 1, 2, 0] == (8 + 3) + 16 * (8 + 2)
    assert c[1][1, 0, 6] == 0.5 and c[3][1, 0, 6] == 0.25
    assert sum(int((a != 0).sum()) for a in (c[1], c[3])) == 2 and (c[2][:, :, [0, 2, 3]] == 0).all()


def test_oracle_attention_by_hand():
    k = np.zeros((3, 1, 2))
    k[:, 0, 0] = [0.0, np.log(2.0), np.log(5.0)]
    v = np.array([[[1.0, -1.0]], [[2.0, 0.0]], [[4.0, 8.0]]])
    q = np.zeros((2, 2, 2))
    q[:, 0, 0] = 1.0
    out, lse, mag, out_off, lse_off = cache.attention(q, k, v, 1.0, True, lambda i, j, s: 0.1 * (s > 1))
    assert np.allclose(out[1, 0], [(1 + 4 + 20) / 8, (-1 + 40) / 8]) and np.allclose(lse[1, 0], np.log(8.0))
    assert np.allclose(out[0, 0], [5 / 3, -1 / 3]) and np.allclose(mag[0, 0], [5 / 3, 1 / 3])
    assert np.allclose(out[0, 1], [1.5, -0.5]) and np.allclose(out[1, 1], [7 / 3, 7 / 3])
    # the token of score ln 5 may be off by a tenth
    assert np.allclose(lse_off[1, 0], 0.1 * 5 / 8) and np.allclose(out_off[1, 0], 0.1 * 5 / 8 * (np.array([4, 8]) + mag[1, 0]))
    assert not out_off[0].any()
    # more queries than tokens: the first see nothing
    out, lse = cache.attention(np.ones((5, 2, 2)), k, v, 1.0, True)[:2]
    assert not out[:2].any() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    assert np.isfinite(cache.attention(np.ones((5, 2, 2)), k, v, 1.0, False)[1]).all()
