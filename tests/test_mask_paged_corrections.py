"""Host-side checks of the masked and the paged attention where they once went wrong."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_context_attention_gb300", "csrc")


def _native(tmp_path, name):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / name
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, os.path.join(HERE, "native", name + ".cpp"), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_capped_scores_keep_their_own_precision(tmp_path):
    """A capped score is off by a part of itself, not of a large cap."""
    _native(tmp_path, "score_cap_relative")


def test_plan_stays_within_its_bounds(tmp_path):
    """Starts that fall by so much that the groups' sum passes 32 bits, windows up to the largest number before
    position 0, and anything else."""
    _native(tmp_path, "paged_plan")


def test_data_of_the_launch_before_is_read_by_plain_loads():
    """A kernel that starts while the launch before it runs waits, then reads what that launch wrote; the read-only path
    would ask for data that is constant from its start on."""
    written = {"attn_bwd.cu": ("tiles", "mask.bad"), "attn_fwd.cu": ("tiles",), "mask_fwd.cu": ("tiles", "v_amax"),
               "v16.cuh": ("shares", "amax"), "paged_attn.cu": ("a.groups", "a.prefix", "a.count")}
    for name, fields in written.items():
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for call in re.finditer(r"__ldg\(([^;]*);", text):
            for field in fields:
                assert not re.search(rf"\b{re.escape(field)}\b", call.group(1)), f"{name}: {call.group(0)}"
