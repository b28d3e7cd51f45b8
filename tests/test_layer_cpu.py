"""The layer entry points (norm_residual_quant, moe_route_topk,
moe_w8a8_block) without a GPU: every call fails its argument checks or is a
no-op, so no kernel launches; and pins of their 64-bit oracle by hand-worked
values."""

import ctypes

import numpy as np
import pytest

import w8a8_int8_quantized_amd as w8
from oracle import layer

OK, ENULL, ESHAPE, EALIGN, EDTYPE, EWS, EVAL = 0, -1, -2, -3, -4, -6, -8
P = ctypes.c_void_p(1 << 20)          # aligned fake address, never dereferenced
P4 = ctypes.c_void_p((1 << 20) + 4)
P2 = ctypes.c_void_p((1 << 20) + 2)
N = ctypes.c_void_p(0)
BF, FP, B, C = w8.W8_BF16, w8.W8_FP32, w8.W8_SCHEME_BLOCK, w8.W8_SCHEME_CHANNEL


def _norm(y=P, res=P, post=P, gate=P, gate_rows=1, scale=1.0, pre=P, eps=1e-6, dtype=BF, scheme=B, M=4, K=256, h=P,
          z=P, q=P, s=P):
    return w8.lib.norm_residual_quant(y, res, post, gate, gate_rows, scale, pre, eps, dtype, scheme, M, K, h, z, q, s,
                                      N)


def test_norm_argument_checks():
    assert _norm(dtype=FP) == EDTYPE and _norm(scheme=2) == EDTYPE
    assert _norm(K=100) == ESHAPE and _norm(M=-1) == ESHAPE and _norm(K=0) == ESHAPE
    assert _norm(K=32768 + 128) == ESHAPE
    assert _norm(gate_rows=2) == ESHAPE and _norm(gate_rows=0) == ESHAPE
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert _norm(eps=eps) == EVAL
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert _norm(scale=scale) == EVAL
    for name in ("y", "pre", "h", "s"):
        assert _norm(**{name: N}) == ENULL, name
    assert _norm(z=N, q=N) == ENULL                    # nothing to write beside h
    for name in ("y", "res", "post", "gate", "pre", "h", "z", "q"):
        assert _norm(**{name: P4}) == EALIGN, name
    assert _norm(s=P2) == EALIGN
    assert _norm(M=0, y=N, pre=N, h=N, z=N, q=N) == OK
    assert w8.lib.w8_status_string(EVAL) != b"unknown status"


def _route(logits=P, dtype=FP, bias=P, score=0, T=4, E=16, topk=2, n_group=4, topk_group=2, group_top=2, scale=1.0,
           ids=P, w=P):
    return w8.lib.moe_route_topk(logits, dtype, bias, score, T, E, topk, n_group, topk_group, group_top, 1, scale, ids,
                                 w, N)


def test_route_argument_checks():
    assert _route(dtype=w8.W8_I32) == EDTYPE and _route(score=2) == EDTYPE
    assert _route(T=-1) == ESHAPE and _route(E=0) == ESHAPE and _route(E=1028, n_group=4) == ESHAPE
    assert _route(topk=0) == ESHAPE and _route(topk=65, E=1024, topk_group=4) == ESHAPE
    assert _route(topk=9) == ESHAPE                    # two groups of four stay
    assert _route(n_group=3) == ESHAPE and _route(n_group=0) == ESHAPE
    assert _route(E=1024, n_group=128) == ESHAPE
    assert _route(topk_group=5) == ESHAPE and _route(topk_group=0) == ESHAPE
    assert _route(group_top=3) == EVAL and _route(scale=float("nan")) == EVAL
    assert _route(logits=N) == ENULL and _route(ids=N) == ENULL and _route(w=N) == ENULL
    assert _route(logits=P2) == EALIGN and _route(ids=P2) == EALIGN and _route(bias=P2) == EALIGN
    assert _route(T=0, logits=N, ids=N, w=N) == OK


def _moe(A=P, sa=P, ids=P, wt=P, w13=P, s13=P, w2=P, s2=P, Y=P, dtype=BF, T=4, topk=2, E=8, I=256, K=256, ws=P,
         nbytes=1 << 40):
    return w8.lib.moe_w8a8_block(A, sa, ids, wt, w13, s13, w2, s2, Y, dtype, T, topk, E, I, K, ws, nbytes, N)


def test_moe_argument_checks():
    assert _moe(dtype=w8.W8_I32) == EDTYPE and _moe(dtype=w8.W8_FP16) == EDTYPE
    assert _moe(T=65) == ESHAPE and _moe(T=-1) == ESHAPE
    assert _moe(topk=0) == ESHAPE and _moe(topk=17) == ESHAPE
    assert _moe(E=0) == ESHAPE and _moe(E=4097) == ESHAPE
    assert _moe(I=0) == ESHAPE and _moe(I=100) == ESHAPE and _moe(I=(1 << 15) + 128) == ESHAPE
    assert _moe(K=0) == ESHAPE and _moe(K=100) == ESHAPE and _moe(K=(1 << 15) + 128) == ESHAPE
    assert _moe(E=4096, I=1 << 15, K=1 << 15) == ESHAPE
    for name in ("A", "sa", "ids", "wt", "w13", "s13", "w2", "s2", "Y", "ws"):
        assert _moe(**{name: N}) == ENULL, name
    for name in ("A", "w13", "w2", "Y", "ws"):
        assert _moe(**{name: P4}) == EALIGN, name
    for name in ("sa", "ids", "wt", "s13", "s2"):
        assert _moe(**{name: P2}) == EALIGN, name
    need = w8.lib.moe_workspace_bytes(4, 2, 256, 256)
    assert need > 4 * 2 * (256 + 4 * 2)
    assert _moe(nbytes=need - 1) == EWS
    assert _moe(T=0, A=N, Y=N, ws=N, nbytes=0) == OK
    assert w8.lib.moe_workspace_bytes(65, 2, 256, 256) == ESHAPE
    assert w8.lib.moe_workspace_bytes(4, 2, 200, 256) == ESHAPE
    assert w8.lib.moe_workspace_bytes(4, 2, 256, 200) == ESHAPE


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(w8.W8Error):
        w8.norm_residual_quant(x, x[0])
    with pytest.raises(w8.W8Error):
        w8.moe_route_topk(torch.zeros(4, 8), 2)


# ------------------------------------------------------------------ oracle
def test_oracle_norm_by_hand():
    y = np.array([[3.0, 4.0, 0.0, 0.0]])
    # mean square 25 / 4 -> rms 2.5
    assert np.allclose(layer.rms_norm(y, np.array([1.0, 2.0, 1.0, 1.0]), eps=0.0), [[1.2, 3.2, 0.0, 0.0]])
    h, t = layer.norm_h(y, residual=np.array([[1.0, 1.0, 1.0, 1.0]]), post_weight=np.ones(4), gate=np.full(4, 0.5),
                        residual_scale=2.0, eps=0.0)
    assert np.allclose(t, [[1.2, 1.6, 0.0, 0.0]]) and np.allclose(h, [[2.2, 2.6, 1.0, 1.0]])


def test_oracle_route_by_hand():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w = layer.route_topk(l, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]])
    ids, w = layer.route_topk(l, 2, renormalise=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    # ties to the lower index; a masked expert is never chosen; slots left over
    ids, w = layer.route_topk(np.array([[0.0, 0.0, -np.inf, 0.0], [np.nan, -np.inf, -np.inf, 1.0]]), 3)
    assert ids.tolist() == [[0, 1, 3], [3, -1, -1]] and np.allclose(w[1], [1, 0, 0])
    # groups (0, 1), (2, 3): the best single expert is in the group of the smaller sum
    l = np.array([[0.0, 3.0, 2.0, 2.0]])
    s = 1 / (1 + np.exp(-l[0]))
    assert s[0] + s[1] < s[2] + s[3]
    assert layer.route_topk(l, 1, sigmoid=True, n_group=2)[0].tolist() == [[2]]
    assert layer.route_topk(l, 1, sigmoid=True, n_group=2, group_top=1)[0].tolist() == [[1]]
    # the bias moves the choice and not the weight
    ids, w = layer.route_topk(l, 1, sigmoid=True, bias=np.array([1.0, 0, 0, 0]), renormalise=False)
    assert ids.tolist() == [[0]] and np.allclose(w, [[0.5]])


def test_oracle_moe_is_the_plain_product():
    """One token, one expert, identity-like weights: gate and up are the
    token's values, the output is quant(silu(x) x)."""
    K = I = 128
    A = np.zeros((1, K), np.int8)
    A[0, :4] = [127, -127, 64, 1]
    w13 = np.zeros((1, 2 * I, K), np.int8)
    w13[0, :I][np.arange(I), np.arange(I)] = 1
    w13[0, I:][np.arange(I), np.arange(I)] = 1
    w2 = np.zeros((1, K, I), np.int8)
    w2[0][np.arange(K), np.arange(I)] = 1
    one = np.ones((1, 1), np.float32)
    x = A[0] / 32.0
    y, tol = layer.moe_block(A, one / 32, np.array([[0]]), np.array([[0.5]]), w13, np.ones((1, 2, 1)), w2,
                             np.ones((1, 1, 1)))
    want = 0.5 * x / (1 + np.exp(-x)) * x
    step = np.abs(want).max() / 127
    assert np.abs(y[0] - want).max() <= step / 2 * (1 + 1e-6) and (y[0][4:] == 0).all()
    assert (tol[0][:4] <= 2 * step).all()
    # an id without an expert adds nothing
    y0, _ = layer.moe_block(A, one, np.array([[-1, 1]]), np.array([[np.nan, np.nan]]), w13, np.ones((1, 2, 1)), w2,
                            np.ones((1, 1, 1)))
    assert not y0.any()
