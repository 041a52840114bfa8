"""The masked and the paged attention where a loose tolerance would hide a fault: caps
far above the scores.

Tolerances as in test_gpu_mask_attn and test_gpu_paged_attn but for the cap's part: a
capped logit is off by at most 2^-19 of itself (caps above 64), |logit| <= min(L, cap), so dx = (d + 4)
2^-24 L + 2^-19 min(L, cap), and its slope 1 - t^2, t = logit / cap, by at most g =
2 t (2^-19 t + dx / cap) + 2^-23.
"""
import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import mask as omask
from tests.helpers import to64
from tests.test_gpu_mask_attn import _run, _sees, _within
from tests.test_gpu_paged_attn import _Setup

pytestmark = pytest.mark.gpu


def _errors(t, d, cap):
    """(e, f, g): the factors of P, of the backward's sums, of them without the cap's slope."""
    L = t["logit"].max(initial=0)
    least = min(L, cap) if cap else L
    dx = (d + 4) * 2.0 ** -24 * L + (2.0 ** -19 * least if cap else 0.0)
    e = 2 * (dx + 2.0 ** -21 + 2.0 ** -23 * least)
    assert e < 2.0 ** -9, "a tolerance that says nothing"
    s = least / cap if cap else 0.0
    g = 2 * s * (2.0 ** -19 * s + dx / cap) + 2.0 ** -23 if cap else 0.0
    return e, 2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -14, g


def _check_rows(t, d, cap, o, lse, dq=None, dk=None, dv=None):
    """Rows of the outputs against the oracle's, those that are given."""
    e, f, g = _errors(t, d, cap)
    _within("O", o, t["o"], 2.0 ** -8 * np.abs(t["o"]) + (2.0 ** -11 + e + 2.0 ** -16) * t["abs_o"])
    some = np.isfinite(t["lse"])
    _within("LSE", lse, t["lse"], np.where(some, e + 2.0 ** -22 * np.abs(np.where(some, t["lse"], 0)), 0))
    for nm, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        if got is not None:
            _within(nm, got, t[nm], 2.0 ** -8 * np.abs(t[nm]) + f * t["abs_" + nm] + g * t["flat_" + nm])


@pytest.mark.parametrize("cap", [1000.0, 2000.0, 1e5, 2.0 ** 20])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_far_above_the_scores(cuda_device, d, cap):
    """The capped logits are then the scores, to their own precision; a query whose scores pass the cap, in the middle
    of a warp, leaves its neighbours theirs."""
    w = inputs.Workload("cap", 400, 4, 2, d, 1, 1, 1, 1, True, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    for far in (False, True):
        if far:
            x["q"][0, 77] *= 2.0 ** 22
        o, lse, dq, dk, dv = _run(w, x, None, cap)
        near = [i for i in range(400) if not far or i != 77]
        # the far query's own logits are too large for a bound that says anything: without its row, its part of dK and dV
        y = {n: to64(t[0]) for n, t in x.items()}
        see = _sees(w, None, 0)[near]
        t = omask.forward_backward(y["q"][near], y["k"], y["v"], y["do"][near], see, ops.default_scale(d), cap,
                                   terms=True)
        _check_rows(t, d, cap, o[0, near], lse[0][:, near], dq[0, near], *((None, None) if far else (dk[0], dv[0])))
        if far:
            assert bool(torch.isfinite(o.float()).all() & torch.isfinite(lse).all())
        elif cap == 2.0 ** 20:   # tanh differs from its argument by less than 2^-24 of it up to 2^-12, that is 256
            o2, lse2, dq2, dk2, dv2 = _run(w, x, None, 0.0)
            _check_rows(t, d, 0.0, o2[0], lse2[0], dq2[0], dk2[0], dv2[0])
            assert (lse - lse2).abs().max() <= 2.0 ** -20 * (1 + lse2.abs().max())


@pytest.mark.parametrize("cap", [1000.0, 2000.0, 1e5, 2.0 ** 20])
@pytest.mark.parametrize("name", ["tokens-ragged", "chunk", "chunk-d64"])
def test_caps_far_above_the_scores_paged(cuda_device, name, cap):
    s = _Setup(name)
    s.cap = cap
    o, lse = s.run()
    assert ops.loong_get_device_status() == ops.LOONG_OK
    at = 0
    for b, (n, new) in enumerate(s.seqs):
        i = np.arange(n - new, n)
        t = omask.forward_backward(to64(s.q[at:at + new]), to64(s.ks[b]), to64(s.vs[b]), None,
                                   omask.sees(np.stack([0 * i, i + 1], 1), n, False), ops.default_scale(s.d), cap,
                                   terms=True)
        e = _errors(t, s.d, cap)[0]
        _within(f"O of sequence {b}", o[at:at + new], t["o"],
                2.0 ** -8 * np.abs(t["o"]) + (2 * (2.0 ** -8 + e) + 2.0 ** -16) * t["abs_o"])
        _within(f"LSE of sequence {b}", lse[:, at:at + new], t["lse"], e + 2.0 ** -22 * (1 + np.abs(t["lse"])))
        at += new


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30, 900])
def test_wide_windows_before_the_first_position(cuda_device, window):
    """More new tokens than a sequence's length holds: those that stand before position 0 see nothing, the others what
    they see without a window."""
    s = _Setup("whole-prompts")
    want = s.run()
    s.window = window
    assert all(torch.equal(a, b) for a, b in zip(s.run(append=False), want))
    s.check(*want)
    short = 40   # the last sequence has 300 new tokens and now a length of 40
    s.lens[2] = short
    o, lse = s.run(append=False)
    assert ops.loong_get_device_status() == ops.LOONG_ERR_DEVICE_CHECK
    at = int(s.starts[3])
    assert bool((o[at - 300:at - short] == 0).all()) and bool(torch.isneginf(lse[:, at - 300:at - short]).all())
    i = np.arange(short)
    t = omask.forward_backward(to64(s.q[at - short:at]), to64(s.ks[2][:short]), to64(s.vs[2][:short]), None,
                               omask.sees(np.stack([0 * i, i + 1], 1), short, False), ops.default_scale(s.d), 0.0,
                               terms=True)
    e = _errors(t, s.d, 0.0)[0]
    _within("O", o[at - short:at], t["o"], 2.0 ** -8 * np.abs(t["o"]) + (2 * (2.0 ** -8 + e) + 2.0 ** -16) * t["abs_o"])
    _within("LSE", lse[:, at - short:at], t["lse"], e + 2.0 ** -22 * (1 + np.abs(t["lse"])))
