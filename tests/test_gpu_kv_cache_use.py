"""Uses of the quantised cache that its allowed arguments include: scales of
either sign, pages that sequences share, keys given once for all tokens, one
workspace and one graph for several lengths."""

import pytest
import torch

import w8a8_int8_quantized_amd as w8
from test_gpu_kv_cache import BF, DEV, FP, WIDE, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spare", [1, WIDE])
@pytest.mark.parametrize("scale", [-0.1, 0.0, -1e-20])
@pytest.mark.parametrize("G,dt", [(2, BF), (8, FP), (24, BF)])
def test_scales_of_either_sign(G, dt, scale, spare):
    p = Problem([(1, 33), (3, 100), (5, 5)], 2 * G, 2, 128, 4, 32, dt, seed=G, spare=spare)
    out, lse = p.call(scale=scale, lse=True)
    p.check(out, lse, scale=scale)


@pytest.mark.parametrize("spare", [1, WIDE])
def test_sequences_that_share_their_pages(spare):
    """The same row of the block table twice (a common beginning): each as by itself, bit for bit."""
    p = Problem([(1, 150), (1, 150)], 8, 2, 128, 4, 32, BF, seed=5, spare=spare)
    table = torch.tensor(p.table, dtype=torch.int32, device=DEV)
    table[1] = table[0]
    q = p.q.to(DEV)
    q[1] = q[0]
    out = p.call(q=q, table=table)
    assert torch.equal(out[0], out[1])
    p.q = q.cpu()
    p.check(out, only=[0])


@pytest.mark.parametrize("bits", [4, 8])
def test_one_key_for_all_tokens(bits):
    """A stride of zero between tokens writes what the copied rows write."""
    g = torch.Generator().manual_seed(bits)
    x = torch.randn(1, 3, 64, generator=g).to(BF).to(DEV)
    slots = torch.tensor([5, 0, 31, 17, 18], dtype=torch.int32, device=DEV)
    got, want = (w8.kv_cache_empty(2, 3, 16, 64, bits=bits) for _ in range(2))
    for c in (got, want):
        for a in c:
            a.zero_()
    row = x.expand(5, 3, 64)
    w8.quant_kv_cache(row, row, slots, got)
    w8.quant_kv_cache(row.contiguous(), row.contiguous(), slots, want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("spare", [1, WIDE])
def test_a_graph_over_lengths_that_change(spare):
    """A captured call replayed with other lengths, eager calls with its workspace between the replays."""
    p = Problem([(1, 130), (1, 257), (1, 64)], 8, 2, 128, 4, 32, BF, seed=9, spare=spare)
    i32 = {"dtype": torch.int32, "device": DEV}
    table, lens, q = torch.tensor(p.table, **i32), torch.tensor([130, 257, 64], **i32), p.q.to(DEV)
    ws = torch.empty(w8.attn_workspace_bytes(1, 8, 2, 128), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    kw = {"ragged": False, "q": q, "table": table, "lens": lens, "workspace": ws}
    p.call(**kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.call(out=out, **kw)
    for new in ([130, 257, 64], [1, 0, 33], [130, 31, 64], [0, 0, 0], [129, 256, 2]):
        lens.copy_(torch.tensor(new, **i32))
        want = p.call(**kw)
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), new
        assert all(not out[b].any() for b, n in enumerate(new) if n == 0)
