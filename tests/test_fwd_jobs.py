"""The forward's score buffers against the order of its matrix instructions
(fwd_jobs.h): a wait that tells two neighbouring phases of a barrier apart by
one bit must never see three.  The check is a host program."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_context_attention_gb300", "csrc")


def test_scores_prove_the_product_two_tiles_back(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "fwd_jobs"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", "fwd_jobs.cpp"), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    assert ", 0 open" in r.stdout
