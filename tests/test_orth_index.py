"""The scaling pass of an orthogonalised update reads every element of a matrix and none outside it, checked on the host (no
GPU) from the index function that the kernel itself uses."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_scaling_pass_stays_inside_the_matrix(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "orth_index_check"
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "sub_bit_weight_b200", "csrc"),
                    os.path.join(ROOT, "tests", "orth_index_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert "orth index ok" in r.stdout
