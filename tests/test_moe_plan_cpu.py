"""CPU checks of the few-token experts' launch rules (csrc/moe_plan.h): what
the kernels take for granted (LDS, grids, columns in one block of the weights)
holds over the sizes the call takes, and the cases of moe_forms.py reach every
form that a size can reach."""

import os
import subprocess

import pytest

import moe_forms

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "moe_plan_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-o", exe, os.path.join(HERE, "moe_plan_check.cpp")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(*args, text=""):
        r = subprocess.run([exe, *args], input=text, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.split("\n")[:-1]

    return run


def test_every_form_has_a_case(plan):
    reachable = set(plan())
    lines = plan("cases", text="".join("%d %d %d %d %d\n" % c[:5] for c in moe_forms.CASES))
    reached = set()
    for c, line in zip(moe_forms.CASES, lines):
        want = ["gate " + c[6], "down " + c[7], "places " + c[8]]
        assert line.split(",") == want, c
        reached.update(want)
    assert reached == reachable, reachable ^ reached


def test_rows_pass_the_fragments():
    """Every gate_up form with experts of up to 16 rows and with one of several passes; every
    down form with several units to an expert where its fragments are fewer than a call's rows."""
    gate, down = {}, {}
    for c in moe_forms.CASES:
        rows = moe_forms.most_rows(moe_forms.ids_of(c), c[2])
        gate.setdefault(c[6], []).append(rows)
        down.setdefault(c[7], []).append(rows)
    for form, rows in gate.items():
        assert max(rows) > 16 * int(form.split()[0]) and (min(rows) <= 16 or form == "4 2 4"), (form, rows)
    for form, rows in down.items():
        assert max(rows) > 16 * int(form.split()[1]), (form, rows)
