"""Batches of many sequences over the quantised cache, against the 64-bit
oracle (tolerances: test_gpu_kv_cache.py)."""

import numpy as np
import pytest
import torch

import w8a8_int8_quantized_amd as w8
from test_gpu_kv_cache import BF, DEV, FORMS, FP, WIDE, Problem
from test_gpu_kv_cache_range import Exact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [BF, FP])
def test_one_piece_among_many_single_tokens_over_a_wide_table(dt):
    """The batch times the piece times the table's width would pass 2^31 units; all tokens together do not."""
    rng = np.random.default_rng(4)
    lens = [(1, int(n)) for n in rng.integers(1, 300, 299)]
    lens.insert(17, (1024, 1100))
    p = Problem(lens, 8, 2, 128, 4, 512, dt, seed=4, spare=6000)
    tiles = p.table.shape[1] * 512 // 32
    assert 300 * 2 * 256 * tiles > 1 << 31
    out, lse = p.call(lse=True)
    p.check(out, lse, sample=12)
    # starts that give every other sequence all rows: more units than are counted, and nothing is computed
    T = p.q.shape[0]
    assert 150 * 2 * (T * 4 // 32) * (tiles - T // 32) > 1 << 32
    starts = torch.tensor([0, T] * 150 + [0], dtype=torch.int32, device=DEV)
    far = torch.full((300,), 2 ** 31 - 1, dtype=torch.int32, device=DEV)
    kept = torch.full_like(out, 7.5)
    p.call(out=kept, q_starts=starts, max_q=T, lens=far)
    assert (kept == 7.5).all()
    assert torch.equal(p.call(), out)


def test_a_table_without_pages():
    """Nothing to see for more sequences than have a workgroup each: zeros."""
    B = 700
    c = w8.kv_cache_empty(1, 2, 16, 64)
    q = torch.randn(B, 8, 64, device=DEV).to(BF)
    table = torch.empty(B, 0, dtype=torch.int32, device=DEV)
    lens = torch.arange(B, dtype=torch.int32, device=DEV)
    out, lse = w8.attn_kv_cache(q, c, table, lens, lse=True)
    assert not out.any() and torch.isneginf(lse).all()


def test_no_query_tokens_to_a_sequence():
    """max_q = 0 leaves nothing of q to compute: refused, but where there is nothing anyway."""
    c = w8.kv_cache_empty(3, 2, 16, 128)
    q = torch.zeros(4, 8, 128, dtype=BF, device=DEV)
    i = torch.zeros(5, dtype=torch.int32, device=DEV)
    with pytest.raises(w8.W8Error):
        w8.attn_kv_cache(q, c, i[:2].view(1, 2), i[:1], q_starts=i[:2], max_q=0)
    assert w8.attn_kv_cache(q[:0], c, i[:2].view(1, 2), i[:1], q_starts=i[:2], max_q=0).shape == (0, 8, 128)
    assert w8.attn_kv_cache(q[:0], c, i[:2].view(1, 2), i[:1], q_starts=i[:2]).shape == (0, 8, 128)


def _batch(seed):
    """40 sequences, of which a few are long: 160 segments of four key heads, joined in order."""
    rng = np.random.default_rng(seed)
    lens = [int(n) for n in rng.integers(0, 60, 34)] + [2000, 1999, 1700, 33, 901, 2017]
    rng.shuffle(lens)
    # 16 units to a segment beside its tiles, and 512 workgroups: the long ones have several followers
    units = sum(4 * (16 + max(1, -(-n // 32))) for n in lens)
    assert 4 * len(lens) * 4 > 512 and units // 512 + 1 < 20
    return lens


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("D,bits", FORMS)
@pytest.mark.parametrize("G", [3, 4, 6])
def test_single_tokens_joined_in_order(G, D, bits, dt):
    """Row tiles of 4 and 8: a full decode batch, a wide table."""
    p = Problem([(1, n) for n in _batch(G)], 4 * G, 4, D, bits, 32, dt, seed=D + G, spare=WIDE)
    out, lse = p.call(lse=True)
    print("share of the tolerance", p.check(out, lse))
    assert all(torch.equal(a, b) for a, b in zip(p.call(lse=True), (out, lse)))


@pytest.mark.parametrize("D,bits,dt", [(64, 8, BF), (128, 4, FP), (256, 4, BF)])
@pytest.mark.parametrize("f", [2.0, 2.0 ** 60])
def test_far_scores_joined_in_order(D, bits, dt, f):
    """Rows that hold their lifts apart, in pieces."""
    p = Exact([max(n, 1) for n in _batch(3)], 1, 4, 4, D, bits, dt, f, seed=2, spare=WIDE)
    p.check(*p.call(True), causal=True, sample=0)
