"""The norms, the router and the few-token experts of a layer, in 64 bits.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Plain numpy float64 from the formulas of include/w8a8.h.  Where the formula
itself rounds (the quantiser's codes and fp32 scales) the rounding is made
here too; nothing else is rounded.
"""

import numpy as np

GROUP = 128
U32 = 2.0 ** -24          # half a step of fp32, relative


def norm_h(y, residual=None, post_weight=None, gate=None, residual_scale=1.0, eps=1e-6):
    """h before its rounding and t = residual_scale * gate * n, both float64 [M, K]."""
    t = y.astype(np.float64)
    if post_weight is not None:
        t = t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * post_weight
    if gate is not None:
        t = t * gate
    t = t * residual_scale
    return (t if residual is None else t + residual), t


def rms_norm(h, weight, eps=1e-6):
    """h rsqrt(mean(h^2) + eps) weight, float64."""
    h = h.astype(np.float64)
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


def route_topk(logits, topk, bias=None, sigmoid=False, n_group=1, topk_group=1, group_top=2, renormalise=True,
               scale=1.0):
    """ids int32 and weights float64 [T, topk], one token and one choice at a time."""
    T, E = logits.shape
    per = E // n_group
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        l = np.minimum(logits[t].astype(np.float64), float(np.finfo(np.float32).max))
        live = l > -np.inf                        # False for NaN too
        if sigmoid:
            with np.errstate(over="ignore", invalid="ignore"):
                s = np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0)
        else:
            s = np.zeros(E)
            if live.any():
                s[live] = np.exp(l[live] - l[live].max())
                s /= s.sum()
        c = np.where(live, s + (bias.astype(np.float64) if bias is not None else 0.0), -np.inf)
        if n_group > 1:
            score = []
            for g in range(n_group):
                v = sorted(c[g * per:(g + 1) * per], reverse=True)[:group_top]
                score.append(sum(x for x in v if x > -np.inf) if v[0] > -np.inf else -np.inf)
            keep = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            for g in range(n_group):
                if g not in keep:
                    c[g * per:(g + 1) * per] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:topk]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[order]
        if renormalise and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def _block_product(a, sa, w, sw):
    """Block-wise product of float64 codes a [n, K], w [N, K] and the sum of its terms' magnitudes."""
    n, K = a.shape
    N = w.shape[0]
    y, mag = np.zeros((n, N)), np.zeros((n, N))
    for kb in range(K // GROUP):
        k = slice(kb * GROUP, (kb + 1) * GROUP)
        p = (a[:, k] @ w[:, k].T) * sa[:, kb:kb + 1] * np.repeat(sw[:, kb], GROUP)[None, :N]
        y += p
        mag += np.abs(p)
    return y, mag


def moe_block(A, sa, ids, weights, w13, s13, w2, s2):
    """The layer's output [T, K] in float64 and how far an fp32 evaluation of
    the same formula may be from it, before its last rounding.

    The bound follows the fp32 steps: a block-wise sum of B exact products
    rounds the scale product, each term and each addition, (B + 3) half steps
    of the terms' magnitudes at most; silu(g) u has |silu'| <= 1.1 and at
    most 8 half steps of its own (exp, addition, division, products); a code
    whose quotient lies within the error of a half-integer may be one step
    off; a group's scale is as far off as its largest element.
    """
    T, K = A.shape
    E, I = w13.shape[0], w13.shape[1] // 2
    y, tol = np.zeros((T, K)), np.zeros((T, K))
    KB, IB = K // GROUP, I // GROUP
    f = np.float64
    for t in range(T):
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if e < 0 or e >= E:
                continue
            wt = float(weights[t, j])
            gu, mag = _block_product(A[t:t + 1].astype(f), sa[t:t + 1].astype(f), w13[e].astype(f), s13[e].astype(f))
            err = (KB + 3) * U32 * mag
            g, u, eg, eu = gu[:, :I], gu[:, I:], err[:, :I], err[:, I:]
            with np.errstate(over="ignore"):
                silu = g / (1.0 + np.exp(-g))
            h = silu * u
            eh = 1.1 * eg * np.abs(u) + np.abs(silu) * eu + 1.1 * eg * eu + 8 * U32 * np.abs(h)
            hb, ehb = h.reshape(IB, GROUP), eh.reshape(IB, GROUP)
            amax = np.abs(hb).max(1, keepdims=True)
            s = np.maximum(amax, 1e-10).astype(np.float32).astype(f)
            s = (s / 127.0).astype(np.float32).astype(f)
            rel_s = (ehb.max(1, keepdims=True) / np.maximum(amax, 1e-10)) + 3 * U32
            quot = hb / s
            eq = ehb / s + np.abs(quot) * (rel_s + U32)
            q = np.clip(np.rint(quot), -127, 127)
            unsure = np.abs(np.abs(quot - np.floor(quot)) - 0.5) <= eq
            step = np.where(unsure, 1.0 + np.floor(eq), 0.0)
            o, omag = _block_product(q.reshape(1, I), s.reshape(1, IB), w2[e].astype(f), s2[e].astype(f))
            # the scale error and the unsure codes, through the same products
            aw = np.abs(w2[e].astype(f)) * np.repeat(np.repeat(s2[e].astype(f), GROUP, 0), GROUP, 1)[:K]
            loose = ((step + np.abs(q) * rel_s) * s).reshape(1, I)
            eo = loose @ aw.T + (IB + 3) * U32 * omag
            y[t] += wt * o[0]
            tol[t] += abs(wt) * (eo[0] + (ids.shape[1] + 2) * U32 * (np.abs(o[0]) + eo[0]))
    return y, tol
