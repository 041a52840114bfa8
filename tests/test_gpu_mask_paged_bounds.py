"""The masked and the paged attention where a loose tolerance or a small problem would
hide a fault: caps far above the scores, windows near 2^31, walks long enough for the
backward's flushes, long sequences.

Tolerances as in test_gpu_mask_attn and test_gpu_paged_attn but for the cap's part: a
capped logit is off by at most 2^-19 of itself (caps above 64), |logit| <= min(L, cap), so dx = (d + 4)
2^-24 L + 2^-19 min(L, cap), and its slope 1 - t^2, t = logit / cap, by at most g =
2 t (2^-19 t + dx / cap) + 2^-23.

Bounds per element add every rounding up with one sign: over N terms they grow with N, sums
of random terms with its root, so of 100,000 terms (a key's gradient in a long sequence)
they let everything pass.  There the norms say more: a term is rounded by at most 2^-8
of itself in P, in dS and at the end, each with a sign of its own, so the error's norm is
at most some 3 * 2^-8 / sqrt(3) of the result's, D's and the logits' errors (e < 2^-9)
beside it: 2^-6 of it at most, of O, whose P is in fp16, too.
"""
import os
import re

import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import mask as omask
from tests.helpers import to64
from tests.test_gpu_checked import _library
from tests.test_gpu_mask_attn import _pack, _run, _sees, _unpack, _within
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


def _norms(**pairs):
    for name, (got, want) in pairs.items():
        got = to64(got)
        assert np.isfinite(got).all(), name
        far = np.linalg.norm(got - want)
        assert far <= 2.0 ** -6 * np.linalg.norm(want), f"{name}: {far / np.linalg.norm(want):.3g} of its norm"


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
        # the far query's own logits are too large for a bound to say anything: without its row and its part of dK, dV
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


def _exact_on_gpu(q, k, v, do, see, scale, cap):
    """omask.forward_backward with its terms, of one sequence, by elementary operations in 64 bits on the GPU."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    g = q.shape[1] // k.shape[1]
    out = {n: torch.zeros_like(t) for n, t in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    out |= {a + n: torch.zeros_like(out[n]) for n in list(out) for a in ("abs_", "flat_")}
    out["lse"] = torch.full((q.shape[1], len(q)), -torch.inf, dtype=torch.float64, device=q.device)
    out["logit"] = torch.zeros_like(out["lse"])
    some, used = see.any(1, keepdim=True), see.any(0)
    # what takes no part is 0
    q, do = (t * some[:, None] for t in (q, do))
    k, v = (t * used[:, None, None] for t in (k, v))
    for h in range(q.shape[1]):
        qq, kk, vv, dd = q[:, h], k[:, h // g], v[:, h // g], do[:, h]
        x, slope = scale * (qq @ kk.T), 1.0
        if cap:
            t = torch.tanh(x / cap)
            x, slope = cap * t, 1 - t * t
        x.masked_fill_(~see, -torch.inf)
        m = torch.where(some, x.amax(1, keepdim=True), 0)
        p = torch.exp(x - m)
        l = p.sum(1, keepdim=True)
        p /= torch.where(some, l, 1)
        o = p @ vv
        out["o"][:, h], out["lse"][h] = o, torch.where(some, m + torch.log(l), -torch.inf)[:, 0]
        out["abs_o"][:, h] = p @ vv.abs()
        out["logit"][h] = scale * qq.norm(dim=1) * kk.norm(dim=1).max()
        ds = p * (dd @ vv.T - (dd * o).sum(1, keepdim=True)) * slope
        flat = p * (dd.abs() @ vv.abs().T + (dd.abs() * out["abs_o"][:, h]).sum(1, keepdim=True))
        for pre, a, y, z in (("", ds, kk, qq), ("abs_", flat * slope, kk.abs(), qq.abs()),
                             ("flat_", flat, kk.abs(), qq.abs())):
            out[pre + "dq"][:, h] = scale * (a @ y)
            out[pre + "dk"][:, h // g] += scale * (a.T @ z)
            out[pre + "dv"][:, h // g] += p.T @ (dd.abs() if pre else dd)
    return {n: t.cpu().numpy() for n, t in out.items()}


def test_exact_on_gpu_is_the_oracle(cuda_device):
    w = inputs.Workload("small", 200, 4, 2, 64, 1, 1, 1, 1, True, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    r = ops.document_ranges([[60, 100]], 200)
    see = _sees(w, r, 0)
    got = _exact_on_gpu(*(x[n][0] for n in ("q", "k", "v", "do")), torch.from_numpy(see).cuda(), 0.125, 20.0)
    want = omask.forward_backward(*(to64(x[n][0]) for n in ("q", "k", "v", "do")), see, 0.125, 20.0, terms=True)
    for n, t in got.items():
        assert np.allclose(t, want[n], rtol=1e-9, atol=1e-12), n


# S, hq, d, cap; the blocks that share a key tile
@pytest.mark.parametrize("S,hq,d,cap,splits", [(9984, 16, 64, 0.0, 1), (9984, 16, 128, 30.0, 1),
                                               (8960, 32, 64, 30.0, 2), (8960, 32, 128, 0.0, 2)])
def test_backward_flushes(cuda_device, S, hq, d, cap, splits):
    """Walks so long that dK and dV leave tensor memory twice on the way; the workspace holds NaN before."""
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    w = inputs.Workload("flush", S, hq, 1, d, 1, 1, 1, 1, True, placement=0, causal=False)
    x = inputs.make_inputs(w, device="cuda")
    r = ops.document_ranges([[S - 100]], S, causal=False)
    desc, mask = ops.make_desc(w), ops.make_mask(rc := r.cuda(), cap)
    nbytes = ops.loong_attn_mask_workspace_size(desc, mask, 1)
    tiles = S // 128
    parts = nbytes - up(ops.loong_attn_workspace_size(desc, 1)) - up(16 * tiles) - up(tiles * hq)
    assert parts == (2 * up(splits * S * d * 4) if splits > 1 else 0)
    with open(os.path.join(os.path.dirname(ops.__file__), "csrc", "attn_bwd.cu")) as f:
        flush = int(re.search(r"constexpr int kFlush = (\d+);", f.read()).group(1))
    # the last tile of rows is padding but for 28 of them
    assert tiles * hq // splits > 2 * flush, "this shape does not flush twice"
    o, lse, res = ops.attn_mask_fwd(w, x["q"], x["k"], x["v"], rc, cap)

    def backward():
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
        grads = [torch.full_like(t, float("nan")) for t in (x["q"], x["k"], x["v"])]
        ops.loong_attn_mask_bwd(desc, mask, x["q"], x["k"], x["v"], o, res, lse, x["do"], *grads, ws)
        assert ops.loong_get_device_status() == ops.LOONG_OK
        return grads
    dq, dk, dv = backward()
    with _library(ops.CHECKED_LIB_PATH):
        again = backward()
    assert torch.equal(dk, again[1]) and torch.equal(dv, again[2])
    t = _exact_on_gpu(*(x[n][0] for n in ("q", "k", "v", "do")), torch.from_numpy(_sees(w, r, 0)).cuda(),
                      ops.default_scale(d), cap)
    _check_rows(t, d, cap, o[0], lse[0], dq[0], dk[0], dv[0])
    rows = slice(0, S - 100)
    for at in range(0, S - 100, 1000):   # keys' tiles one after the other, so that none hides behind the rest
        some = slice(at, at + 1000)
        _norms(o=(o[0, rows][some], t["o"][rows][some]), dq=(dq[0, rows][some], t["dq"][rows][some]),
               dk=(dk[0, rows][some], t["dk"][rows][some]), dv=(dv[0, rows][some], t["dv"][rows][some]))


@pytest.mark.parametrize("d,cap", [(64, 25.0), (128, 0.0)])
@pytest.mark.parametrize("layout", [ops.LAYOUT_NATURAL, ops.LAYOUT_RANK_MAJOR])
def test_long_sequence_of_documents(cuda_device, d, cap, layout):
    """131,072 tokens of packed documents up to 9,000 long, every one of them up to the last token: a short document
    whole, of a long one the rows and keys at its end, which see or are seen by rows of it alone."""
    S, hq, hkv = 131072, 4, 2
    w = inputs.Workload("long", S, hq, hkv, d, 2, 8, 4, 2, True)
    x = inputs.make_inputs(w, device="cuda")
    rng = np.random.default_rng(6)
    lengths = []
    while sum(lengths) < S - 1000:
        lengths.append(int(rng.integers(1, 9000)))
    lengths = lengths[:-1]
    r = ops.document_ranges([lengths], S)
    out = _run(w, x if layout == ops.LAYOUT_NATURAL else _pack(w, x), r, cap, layout=layout)
    if layout == ops.LAYOUT_RANK_MAJOR:
        out = [t if i == 1 else _unpack(w, t) for i, t in enumerate(out)]
    o, lse, dq, dk, dv = out
    starts = np.concatenate([[0], np.cumsum(lengths)])
    for a, b in zip(starts[:-1], starts[1:]):
        a, b = int(a), int(b)
        first = max(a, b - 256)   # causal: the keys from here on are seen by the rows from here on alone
        n = b - first
        see = omask.sees(np.tile([0, b - a], (n, 1)), b - a, True, first=first - a)
        t = omask.forward_backward(to64(x["q"][0, first:b]), to64(x["k"][0, a:b]), to64(x["v"][0, a:b]),
                                   to64(x["do"][0, first:b]), see, ops.default_scale(d), cap, terms=True)
        for name in list(t):
            if name[-2:] in ("dk", "dv"):
                t[name] = t[name][first - a:]
        _check_rows(t, d, cap, o[0, first:b], lse[0][:, first:b], dq[0, first:b], dk[0, first:b], dv[0, first:b])
        if n == 256:
            _norms(o=(o[0, first:b], t["o"]), dq=(dq[0, first:b], t["dq"]), dk=(dk[0, first:b], t["dk"]),
                   dv=(dv[0, first:b], t["dv"]))
    pad = int(starts[-1])
    assert bool((o[0, pad:] == 0).all()) and bool(torch.isneginf(lse[0][:, pad:]).all())
    assert all(bool((g[0, pad:] == 0).all()) for g in (dq, dk, dv))
