"""A key/value cache in 4 or 8 bits and attention over it, in 64 bits.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Rows (one token of one head) are quantised by the definition of quant.py and
int4.py with a row as the group; the attention is the formula of
include/w8a8.h on the dequantised rows in float64.
"""

import numpy as np

from .quant import EPS, widen

F32 = np.float32


def quant_rows(x, bits):
    """x [..., D] -> integer codes [..., D] (int32) and fp32 scales [...]."""
    x32 = widen(x)
    top = F32(127.0 if bits == 8 else 7.0)
    s = (np.maximum(np.abs(x32).max(-1), EPS) / top).astype(F32)
    q = np.clip(np.rint((x32 / s[..., None]).astype(F32)), -top, top)
    return q.astype(np.int32), s


def row_bytes(q, bits):
    """Codes [..., D] as bytes [..., D * bits / 8] (uint8)."""
    if bits == 8:
        return q.astype(np.int8).view(np.uint8)
    u = (q + 8).astype(np.uint8)
    return u[..., 0::2] + u[..., 1::2] * np.uint8(16)


def put(cache, page, place, head, kq, ks, vq, vs, bits):
    """One token's rows into numpy arrays (k, k_scale, v, v_scale) laid out as the header says."""
    k, k_scale, v, v_scale = cache
    k[page, head, place] = row_bytes(kq, bits)
    k_scale[page, head, place] = ks
    b = row_bytes(vq, bits)
    n = b.size // 16
    for c in range(16):
        v[page, head, place // 4, c, place % 4] = b[c * n:(c + 1) * n]
    v_scale[page, head, place] = vs


def attention(q, k, v, scale, causal, score_error=None, which=None):
    """One sequence: q [n, Hq, D], k and v [L, Hkv, D] float64.

    Returns out [n, Hq, D], lse [n, Hq], and for tolerances the sum of the
    terms' magnitudes mag = sum p |v| / sum p [n, Hq, D], and how far out and
    lse move at most, in first order, where the score of query (i, j) with
    token t is off by score_error(i, j, s) [seen] at most: p errs by the
    factor of it in numerator and denominator.  which: the queries whose rows
    are computed (all, if None).
    """
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    out, mag, lse = np.zeros((n, Hq, D)), np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    out_off, lse_off = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n) if which is None else which:
        seen = max(0, L - n + i + 1) if causal else L
        if seen == 0:
            continue
        for j in range(Hq):
            h = j // (Hq // Hkv)
            s = scale * (k[:seen, h] @ q[i, j])
            m = s.max()
            p = np.exp(s - m)
            p /= p.sum()
            out[i, j] = p @ v[:seen, h]
            mag[i, j] = p @ np.abs(v[:seen, h])
            lse[i, j] = m + np.log(np.exp(s - m).sum())
            if score_error is not None:
                e = p * score_error(i, j, s)
                lse_off[i, j] = e.sum()
                out_off[i, j] = e @ np.abs(v[:seen, h]) + e.sum() * mag[i, j]
    return out, lse, mag, out_off, lse_off
