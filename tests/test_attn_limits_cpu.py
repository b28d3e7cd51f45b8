"""The largest sizes that attention over a quantised cache takes: its plan
(csrc/attn_plan.h) in C++, and the argument checks, without a GPU (no call
gets past them)."""

import ctypes
import os
import subprocess

import pytest

import w8a8_int8_quantized_amd as w8

HERE = os.path.dirname(os.path.abspath(__file__))
ESHAPE, EWS = -2, -6
P = ctypes.c_void_p(1 << 20)          # aligned fake address, never dereferenced
N = ctypes.c_void_p(0)


def test_the_plan_at_the_largest_sizes(tmp_path):
    exe = str(tmp_path / "attn_limits_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined",
                        "-fno-sanitize-recover=undefined", "-o", exe, os.path.join(HERE, "attn_limits_check.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


def _attn(B, T, max_q, max_pages, Hq=32, Hkv=8, D=128, page=64):
    """Without a workspace: EWS where the sizes pass."""
    return w8.lib.attn_kv_cache(P, w8.W8_BF16, Hq * D, P, P, P, P, P, P, P, B, T, max_q, Hq, Hkv, D, 4, 3, page, max_pages,
                                0.1, 1, P, N, P, 0, N)


@pytest.mark.parametrize("B,n", [(128, 2048), (32, 8192), (600, 1), (256, 1024)])
def test_steps_of_many_pieces(B, n):
    """All of a batch's tokens together count, not the longest piece times the batch: a table for 131072 tokens."""
    assert _attn(B, B * n, n, 2048) == EWS
    assert _attn(B, B * n, B * n, 2048) == EWS           # max_q unknown: all tokens
    assert _attn(B, n + B - 1, n, 2048) == EWS           # one piece, the others single tokens


def test_more_work_than_is_counted():
    """A million sequences over tables for a million tokens each."""
    assert _attn(1 << 20, 1 << 20, 1, 1 << 14) == ESHAPE
    assert _attn(1 << 20, 1 << 20, 1 << 20, 1 << 14) == ESHAPE
