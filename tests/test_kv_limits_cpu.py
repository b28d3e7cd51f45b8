"""The largest sizes and values that the calls on a quantised cache take,
without a GPU: every call fails its argument checks, so no kernel launches."""

import ctypes

import pytest

import w8a8_int8_quantized_amd as w8

ESHAPE, EALIGN, EWS, EVAL = -2, -3, -6, -8
P = ctypes.c_void_p(1 << 20)          # aligned fake address, never dereferenced
P2 = ctypes.c_void_p((1 << 20) + 2)
N = ctypes.c_void_p(0)


def _write(T, H):
    """With slots that no call takes: one whose sizes pass gives EALIGN."""
    return w8.lib.quant_kv_cache(P, P, w8.W8_BF16, 4096, 4096, P2, T, H, 128, 4, 3, 64, P, P, P, P, N)


def _read(T, H):
    return w8.lib.dequant_kv_cache(P, P, P, P, P2, T, H, 128, 4, 3, 64, P, P, w8.W8_BF16, N)


@pytest.mark.parametrize("call", [_write, _read])
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 8, 9, 4096])
def test_rows_of_a_call(call, H):
    """Four heads to a workgroup, whether they are there or not: the lanes of the largest call are 2^31."""
    most = (1 << 27) // ((H + 3) // 4 * 4)
    assert call(most, H) == EALIGN
    assert call(most + 1, H) == ESHAPE
    assert (most + 3) // 4 * ((H + 3) // 4) * 256 < 1 << 32


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.3e38, -3.3e38])
def test_scale_stays_finite_in_base_2(scale):
    """The kernels take scale * log2(e), which has to be finite; 2.3e38 still is."""
    def call(x):
        return w8.lib.attn_kv_cache(P, w8.W8_BF16, 4096, P, P, P, P, P, P, P, 2, 4, 4, 32, 8, 128, 4, 3, 64, 2, x, 1, P,
                                    N, P, 0, N)
    assert call(scale) == EVAL
    assert call(2.3e38) == EWS and call(-2.3e38) == EWS
