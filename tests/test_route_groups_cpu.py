"""CPU check of the router's group arithmetic (csrc/route_groups.h): for every
number of experts and groups, each expert's group is e / (E / n_group), and no
element of a lane, those past the last expert included, shifts the 64-bit word
of the kept groups by 64 or more (129 experts in 43 groups once shifted by up
to 85, undefined in C++).  Built with g++ under UBSan."""

import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_route_groups(tmp_path):
    exe = str(tmp_path / "route_groups_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-o", exe,
                        os.path.join(HERE, "route_groups_check.cpp")], capture_output=True, text=True)
    if r.returncode != 0 and "ubsan" in r.stderr:
        pytest.skip(f"g++ cannot build with -fsanitize=undefined here: {r.stderr[:200]}")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
