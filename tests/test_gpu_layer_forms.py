"""GPU parity of the layer entry points in forms and sizes that
test_gpu_layer.py does not reach, with its oracle, checks and tolerances."""

import pytest
import torch

import w8a8_int8_quantized_amd as w8
from test_gpu_layer import DEV, _check_route, _gen, _norm_inputs, _route, _same

pytestmark = pytest.mark.gpu


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
