"""GPU parity of the layer entry points in forms and sizes that
test_gpu_layer.py does not reach, with its oracle, checks and tolerances."""

import pytest
import torch

from test_gpu_layer import _check_route, _gen, _route

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
