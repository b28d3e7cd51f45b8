"""GPU parity of the layer entry points in forms and sizes that
test_gpu_layer.py does not reach, with its oracle, checks and tolerances."""

import numpy as np
import pytest
import torch

import moe_forms
import w8a8_int8_quantized_amd as w8
from test_gpu_layer import (DEV, _check_moe, _check_norm, _check_route, _gen, _moe_inputs, _norm_inputs, _route,
                            _same, _to)

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- norm
# More than 256 rows, so that each of the launch shapes for many rows is taken:
# threads x chunks 256 x 1, 256 x 2, 512 x 2, 512 x 3, 512 x 4, and with the
# later loads 1024 x 3 and 1024 x 4 (a size in each shape's middle or at its
# border).  A thread's squares are at most 32, as the tolerances count.
MANY_ROWS = [1024, 2176, 4224, 8320, 12288, 12416, 16384, 16512, 18432, 24704, 32768]


@pytest.mark.parametrize("scheme", [w8.W8_SCHEME_BLOCK, w8.W8_SCHEME_CHANNEL])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", MANY_ROWS)
def test_norm_many_rows(K, dt, scheme):
    print(f"norm M=257 K={K} {dt} scheme={scheme}", flush=True)
    d = _norm_inputs(257, K, dt, seed=K, gate="token" if scheme == w8.W8_SCHEME_BLOCK else "channel")
    got = w8.norm_residual_quant(**{k: v.to(DEV) for k, v in d.items()}, residual_scale=0.37, eps=1e-5, scheme=scheme,
                                 normed=True)
    _check_norm(d, 0.37, 1e-5, scheme, got, dt)


@pytest.mark.parametrize("K", [8320, 18432, 32768])
@pytest.mark.parametrize("name", ["residual", "y"])
def test_norm_many_rows_in_place(K, name):
    """h into the memory of an input that the later loads read: against the oracle."""
    d = _norm_inputs(257, K, torch.bfloat16, seed=K + 1)
    g = {k: v.to(DEV) for k, v in d.items()}
    M = 257
    out = (g[name], torch.empty(M, K, dtype=torch.int8, device=DEV), torch.empty(M, K // 128, device=DEV),
           torch.empty(M, K, dtype=torch.bfloat16, device=DEV))
    got = w8.norm_residual_quant(**g, residual_scale=-0.6, normed=True, out=out)
    assert got[0].data_ptr() == g[name].data_ptr()
    _check_norm(d, -0.6, 1e-6, w8.W8_SCHEME_BLOCK, got, torch.bfloat16)


# ------------------------------------------------------------------ router
@pytest.mark.parametrize("E,n_group", [(192, 64), (129, 43), (576, 64), (65, 5)])
def test_route_lanes_past_the_last_expert(E, n_group):
    """E is no power of two: lanes hold elements past E whose group index would pass the last group."""
    logits = 2 * torch.randn(7, E, generator=_gen(E))
    for sigmoid in (False, True):
        for kept in (1, n_group // 2, n_group):
            kw = dict(sigmoid=sigmoid, n_group=n_group, topk_group=kept, bias=0.1 * torch.randn(E, generator=_gen(3)))
            topk = min(5, kept * (E // n_group))
            _check_route(logits, _route(logits, topk, **kw), topk, **kw)


def test_route_saturated_scores_tie():
    """Scores that 64 bits round to the same number tie, whatever their logits: the lower index, by kernel and oracle."""
    for sigmoid, bias, logits, want in [
            (True, None, [30.0, 38.0, 40.0, 39.0, 200.0], [1, 2, 3, 4]),
            (True, None, [-800.0, -711.0, -30.0, -900.0], [2, 0, 1, 3]),
            (False, None, [0.0, -750.0, -746.0, -747.0], [0, 1, 2, 3]),
            (False, 1.0, [-40.0, -39.0, 0.0, -41.0], [2, 0, 1, 3])]:
        l = torch.tensor([logits])
        b = None if bias is None else torch.full((l.shape[1],), bias)
        got = _route(l, 4, sigmoid=sigmoid, bias=b)
        assert got[0].tolist() == [want]
        _check_route(l, got, 4, sigmoid=sigmoid, bias=b)


# ----------------------------------------------------------------- experts
@pytest.mark.parametrize("case", moe_forms.CASES, ids=lambda c: "x".join(str(v) for v in c[:5]))
def test_moe_forms(case):
    """Every form of the kernels, with experts of many rows among experts of few."""
    print(f"moe {case}", flush=True)
    T, topk, E, I, K = case[:5]
    ids = moe_forms.ids_of(case)
    args = _moe_inputs(T, topk, E, I, K, seed=T + topk + E, ids=ids)
    args[3][ids < 0] = np.nan
    t = _to(args)
    ws = torch.full((w8.moe_workspace_bytes(T, topk, I, K),), 0xFF, dtype=torch.uint8, device=DEV)
    buf = torch.full((T + 1, K), 5.0, device=DEV)
    got = w8.moe_w8a8_block(*t, out=buf[:T], workspace=ws)
    _check_moe(args, got, w8.moe_w8a8_block(*t))
    assert bool((buf[T] == 5).all())


# ------------------------------------------------------------------ binding
def test_public_stream_and_device_calls(monkeypatch):
    """The handle and device that a torch without the private names gives: the
    same stream, so work on a side stream stays in its order."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert w8._public_raw_stream(0) == side.cuda_stream == w8._raw_stream(0)
    d = {k: v.to(DEV) for k, v in _norm_inputs(64, 1024, torch.bfloat16, seed=3).items()}
    want = w8.norm_residual_quant(**d)
    monkeypatch.setattr(w8, "_raw_stream", w8._public_raw_stream)
    monkeypatch.setattr(w8, "_current_device", torch.cuda.current_device)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = w8.norm_residual_quant(**d)
    side.synchronize()
    assert _same(got, want)
