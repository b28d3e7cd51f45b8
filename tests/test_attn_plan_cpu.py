"""CPU check of how attention over a cache is shared out (csrc/attn_plan.h)."""

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_tile_once_and_every_piece_joined(tmp_path):
    exe = str(tmp_path / "attn_plan_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror",
                        "-o", exe, os.path.join(HERE, "attn_plan_check.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
