"""Host-side checks of the masked and the paged attention where they once went wrong."""
import os
import re
import shutil
import subprocess

import pytest
import torch

from head_context_attention_gb300 import inputs, ops

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_context_attention_gb300", "csrc")
W = inputs.WORKLOADS["tiny-gqa-s1k"]
# q, k_pages, v_pages, table, lens, starts: on the host, where a call that is fine so far ends
_PAGED = (torch.zeros(1, 4, 64, dtype=torch.bfloat16), *[torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)] * 2,
          torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


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


@pytest.mark.parametrize("value", [1e-46, -1e-46, 5e-324, 2.0 ** -150])
def test_a_number_that_vanishes_in_single_precision_is_refused(loong_lib, value):
    """0 would stand for no cap, or for the default scale."""
    x = inputs.make_inputs(W)
    with pytest.raises(ValueError, match="score_cap"):
        ops.make_mask(None, value)
    with pytest.raises(ValueError, match="score_cap"):
        ops.attn_mask_fwd(W, x["q"], x["k"], x["v"], score_cap=value)
    for kw in ({"score_cap": value}, {"scale": value}):
        with pytest.raises(ValueError, match=next(iter(kw))):
            ops.paged_attn(*_PAGED, **kw)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 32 + 5])
def test_a_window_beyond_32_bits_is_refused(loong_lib, window):
    """Its low 32 bits would be taken."""
    with pytest.raises(ValueError, match="window"):
        ops.paged_attn(*_PAGED, window=window)


def test_a_window_is_a_whole_number(loong_lib):
    for _ in range(2):
        with pytest.raises(TypeError):
            ops.paged_attn(*_PAGED, window=8.0)
        with pytest.raises(ValueError, match="CUDA device"):
            ops.paged_attn(*_PAGED, window=8)


@pytest.mark.parametrize("window", [12, 13, 2 ** 31 - 13, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("causal", [True, False])
def test_document_ranges_with_a_window_wider_than_any_document(window, causal):
    lengths = [[4, 1, 0, 5], [], [12]]
    assert torch.equal(ops.document_ranges(lengths, 12, window=window, causal=causal),
                       ops.document_ranges(lengths, 12, causal=causal))


def test_document_ranges_with_a_prefix_longer_than_any_document():
    assert torch.equal(ops.document_ranges([[4, 8]], 12, prefix=[[2 ** 40, 2 ** 31]]),
                       ops.document_ranges([[4, 8]], 12, causal=False))


def test_the_smallest_numbers_are_the_library_s_to_judge(loong_lib):
    for value in (2.0 ** -149, 1.01 * 2.0 ** -150):
        assert ops.loong_attn_mask_check(ops.make_desc(W), ops.make_mask(None, value)) == ops.LOONG_ERR_UNSUPPORTED
