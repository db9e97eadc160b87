"""The order of the units of the output layer's loss and gradients, and what
they wait for, checked on the host over many sizes (tests/c/xent_units.cpp walks
the list that the kernel walks)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "deterministic_invariant_gemm_fwd_gb300", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("units") / "xent_units")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "c", "xent_units.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    return exe


def run(program, rule):
    r = subprocess.run([program, rule], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


def test_units_wait_only_for_earlier_ones(program):
    run(program, "order")


def test_waits_imply_what_a_unit_needs(program):
    run(program, "enough")
