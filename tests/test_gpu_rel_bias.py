"""Ring attention with a bucketed relative bias, and its gradients, against the
float64 oracle.

Tolerances, per element, from what rounds on the way (half steps: bf16 2^-8 of
the value, fp16 2^-11, fp32 2^-24):
  * a logit x: products of bf16 are exact, their sum and the bias add take at
    most d + 4 fp32 roundings of at most L = scale |q| |k|max + |bias|max:
    dx = (d + 4) 2^-24 L; the exponential and its argument 2^-21 + 2^-23 L more:
    every P is off by at most a factor 1 + e, e = 2 (dx + 2^-21 + 2^-23 L).
  * O: P rounded to fp16, sums in fp32, O to bf16: 2^-8 |O| + (2^-11 + e + 2^-16) A,
    A = P |V|; LSE: e + 2^-22 |LSE|.
  * the backward's P and dS are rounded to bf16, D comes from O and its residual
    (P to fp16: 2^-11 of A, then 2^-16): dS is off by at most
    f = 2^-8 + 2^-11 + 2 e + 2^-14 of a = P (|dO| |V| + |dO| A), so dQ, dK, dV by f
    times the same sums over absolute values, plus 2^-8 of themselves.
  * dtable does not use the rounded dS: (2^-11 + 2 e + 2^-14) of the sum of a,
    plus 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import bias as obias
from tests.helpers import to64

pytestmark = pytest.mark.gpu

LOG = "log"   # log_buckets(num, max_distance)
# S, hq, hkv, d, hp, cp, inner, zigzag, batch, causal, buckets, table
CASES = {
    "one-token": (1, 2, 1, 64, 1, 1, 1, 0, 1, 1, (LOG, 8, 20), None),
    "two-tokens": (2, 2, 2, 128, 1, 1, 1, 1, 3, 1, (LOG, 8, 20), None),
    "three-keys": (3, 2, 1, 64, 1, 3, 3, 0, 1, 0, (LOG, 8, 20), None),
    "under-a-tile": (100, 4, 2, 64, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), None),
    "tile-and-one": (129, 3, 1, 128, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), None),
    "gqa": (512, 4, 2, 64, 2, 4, 2, 1, 1, 1, (LOG, 32, 128), None),
    "ragged-blocks": (600, 2, 1, 128, 1, 3, 3, 1, 1, 1, (LOG, 16, 300), None),
    "not-causal": (398, 2, 2, 64, 1, 2, 2, 0, 2, 0, (LOG, 32, 128), None),
    "not-causal-d128": (256, 3, 1, 128, 1, 2, 1, 1, 1, 0, (LOG, 16, 60), None),
    "group-of-34": (150, 34, 1, 64, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), None),
    "far-boundaries": (900, 2, 1, 64, 1, 1, 1, 0, 1, 1, (4, [127, 128, 500]), None),
    "tile-boundaries": (640, 2, 1, 128, 1, 1, 1, 0, 1, 1, (5, [128, 256, 384, 512]), None),
    "shared-buckets": (300, 2, 1, 64, 1, 1, 1, 0, 1, 0, (3, [-200, -1, 0, 1, 200], [0, 1, 2, 2, 1, 0]), None),
    "one-bucket": (400, 2, 1, 64, 1, 1, 1, 0, 1, 1, (1, []), None),
    "beyond-all": (300, 2, 1, 64, 1, 1, 1, 0, 1, 1, (3, [-1000, 5000]), None),
    "256-buckets": (520, 2, 2, 128, 1, 1, 1, 0, 1, 1, (256, list(range(1, 256))), None),
    "window": (700, 2, 1, 64, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), "window"),
    "window-d128": (700, 2, 1, 128, 1, 1, 1, 0, 1, 1, (3, [150, 400]), "window"),
    "empty-rows": (300, 2, 1, 64, 1, 1, 1, 0, 1, 1, (4, [20, 40, 200]), "no-near"),
    "empty-rows-ring": (384, 2, 1, 128, 1, 3, 3, 1, 1, 1, (4, [20, 140, 200]), "no-near"),
    "lowest": (300, 2, 1, 64, 1, 1, 1, 0, 1, 0, (4, [-20, 1, 130]), "lowest"),
    "nothing": (140, 2, 1, 64, 1, 1, 1, 0, 1, 1, (1, []), "no-near"),
    "one-head-groups": (600, 3, 3, 128, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), None),
    "one-head-groups-even": (1024, 2, 2, 64, 1, 2, 2, 1, 1, 1, (LOG, 16, 400), None),
    "one-head-not-causal": (513, 2, 2, 128, 1, 1, 1, 0, 2, 0, (LOG, 32, 128), None),
    "groups-of-five": (420, 10, 2, 64, 1, 1, 1, 0, 1, 1, (LOG, 32, 128), None),
    "one-head-window": (900, 2, 2, 64, 1, 1, 1, 0, 1, 1, (3, [150, 400]), "window"),
    "large-bias": (400, 2, 1, 64, 1, 1, 1, 0, 1, 1, (LOG, 16, 300), "large"),
}


def _make(name, seed=0):
    S, hq, hkv, d, hp, cp, inner, zz, B, causal, bk, how = CASES[name]
    w = inputs.Workload(name, S, hq, hkv, d, hp, cp, inner, cp // inner, True, placement=zz, batch=B,
                        causal=bool(causal))
    if bk[0] == LOG:
        buckets = ops.log_buckets(bk[1], bk[2], causal=bool(causal))
    else:
        buckets = ops.RelBuckets(*bk)
    x = inputs.make_inputs(w, device="cuda", seed_offset=seed)
    g = torch.Generator(device="cuda").manual_seed(100 + seed)
    t = torch.randn((buckets.num_buckets, hq), generator=g, device="cuda")
    if how == "large":
        t *= 20
    t = t.to(torch.bfloat16)
    if how == "window":
        t[-1] = -torch.inf
    if how == "no-near":
        t[0] = -torch.inf
    if how == "lowest":
        t[1, 0], t[2, 1] = torch.finfo(torch.bfloat16).min, -2.0 ** 100
    return w, x, t, buckets


def _pack(w, x):
    return {n: ops.headctx_pack(t, w.cp, w.hp, 1 if w.placement else 2) for n, t in x.items()}


def _unpack(w, t):
    return ops.headctx_unpack(t, w.batch, w.cp, w.hp, 1 if w.placement else 2)


def _run(w, x, t, buckets, mode=ops.MODE_FUSED, layout=ops.LAYOUT_NATURAL, res=True):
    o, lse, o_res = ops.attn_bias_fwd(w, x["q"], x["k"], x["v"], t, buckets, mode=mode, layout=layout, res=res)
    grads = ops.attn_bias_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], t, buckets, o_res=o_res, mode=mode,
                              layout=layout)
    assert ops.loong_get_device_status() == ops.LOONG_OK
    return (o, lse) + grads


def _within(name, got, want, tol):
    got = to64(got)
    assert got.shape == want.shape, name
    same_inf = np.isneginf(got) & np.isneginf(want)
    assert np.all(np.isfinite(got) | same_inf), f"{name}: non-finite"
    err = np.where(same_inf, 0, np.abs(np.where(same_inf, 0, got) - np.where(same_inf, 0, want)))
    assert np.all(err <= tol), (f"{name}: {(err > tol).sum()} of {err.size} outside; worst "
                                f"{np.max(err / np.maximum(tol, 1e-300)):.3g} of the tolerance")


def _e(w, r):
    """How far a probability may be off, relative (see the top)."""
    L = r["logit"].max()
    return 2 * ((w.head_dim + 4) * 2.0 ** -24 * L + 2.0 ** -21 + 2.0 ** -23 * L)


def _check(w, x, t, buckets, out):
    o, lse, dq, dk, dv, dt = out
    scale = ops.default_scale(w.head_dim)
    t64 = to64(t)
    t64 = np.where(t64 <= -2.0 ** 100, -np.inf, t64)
    want_dt, tol_dt = np.zeros(t64.shape), np.zeros(t64.shape)
    for b in range(w.batch):
        r = obias.forward_backward(to64(x["q"][b]), to64(x["k"][b]), to64(x["v"][b]), to64(x["do"][b]), t64,
                                   buckets.bounds, buckets.bucket_of, scale, w.causal, terms=True)
        e = _e(w, r)
        _within("O", o[b], r["o"], 2.0 ** -8 * np.abs(r["o"]) + (2.0 ** -11 + e + 2.0 ** -16) * r["abs_o"])
        some = np.isfinite(r["lse"])
        _within("LSE", lse[b], r["lse"], np.where(some, e + 2.0 ** -22 * np.abs(np.where(some, r["lse"], 0)), 0))
        f = 2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -14
        for nm, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            _within(nm, got[b], r[nm], 2.0 ** -8 * np.abs(r[nm]) + f * r["abs_" + nm])
        want_dt += r["dtable"]
        tol_dt += (2.0 ** -11 + 2 * e + 2.0 ** -14) * r["abs_dtable"]
    _within("dtable", dt, want_dt, tol_dt + 2.0 ** -8 * np.abs(want_dt))


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(cuda_device, name):
    w, x, t, buckets = _make(name)
    out = _run(w, x, t, buckets)
    _check(w, x, t, buckets, out)
    # the table's gradient in the same bits again
    assert torch.equal(_run(w, x, t, buckets)[5].view(torch.int16), out[5].view(torch.int16))


@pytest.mark.parametrize("name", list(CASES))
def test_many_sequences(cuda_device, name):
    """Copies of a case's sequences, more than one block per SM: the blocks then hold two heads (or two query tiles of
    one) where the few of the case alone hold one.  A row's arithmetic is the same: the same bits, but dQ's adds, and
    the table's gradient the copies' sum (each rounded to bf16 once, 2^-8 of it)."""
    w, x, t, buckets = _make(name)
    one = _run(w, x, t, buckets)
    copies = 160 // w.hq + 1
    many = w.with_(batch=w.batch * copies)
    out = _run(many, {n: v.repeat(copies, 1, 1, 1) for n, v in x.items()}, t, buckets)
    for i in (0, 1, 3, 4):
        a, b = out[i].unflatten(0, (copies, w.batch)), one[i]
        assert all(torch.equal(c, b) for c in a), i
    a = out[2].unflatten(0, (copies, w.batch))
    assert (a.float() - one[2].float()).abs().max() <= 2.0 ** -7 * one[2].float().abs().max()
    assert torch.all((out[5].float() - copies * one[5].float()).abs() <= 2.0 ** -7 * copies * one[5].float().abs() + 2.0 ** -14 * copies)


@pytest.mark.parametrize("name", ["gqa", "ragged-blocks", "not-causal", "not-causal-d128", "empty-rows-ring", "window",
                                  "one-head-groups-even", "groups-of-five"])
def test_stepwise_matches_oracle(cuda_device, name):
    w, x, t, buckets = _make(name)
    _check(w, x, t, buckets, _run(w, x, t, buckets, mode=ops.MODE_STEPWISE))


@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE, ops.MODE_STEPWISE_COPY, ops.MODE_STEPWISE_COPY_AB])
@pytest.mark.parametrize("name", ["gqa", "empty-rows-ring", "one-head-groups-even"])
def test_ranks_layout(cuda_device, name, mode):
    w, x, t, buckets = _make(name)
    o, lse, dq, dk, dv, dt = _run(w, _pack(w, x), t, buckets, mode=mode, layout=ops.LAYOUT_RANK_MAJOR)
    _check(w, x, t, buckets, (_unpack(w, o), lse, _unpack(w, dq), _unpack(w, dk), _unpack(w, dv), dt))


def test_without_the_residual(cuda_device):
    """D from bf16 O: 2^-8 instead of 2^-11 of A more in dS, and in dtable."""
    w, x, t, buckets = _make("gqa")
    o, lse, dq, dk, dv, dt = _run(w, x, t, buckets, res=False)
    r = obias.forward_backward(to64(x["q"][0]), to64(x["k"][0]), to64(x["v"][0]), to64(x["do"][0]), to64(t),
                               buckets.bounds, buckets.bucket_of, ops.default_scale(w.head_dim), True, terms=True)
    _within("dtable", dt, r["dtable"], 2.0 ** -8 * np.abs(r["dtable"]) + 2.0 ** -7 * r["abs_dtable"])
    _within("dq", dq[0], r["dq"], 2.0 ** -8 * np.abs(r["dq"]) + 2.0 ** -6 * r["abs_dq"])


@pytest.mark.parametrize("d,hq", [(64, 4), (128, 4), (64, 2), (128, 6)])
def test_zero_table_is_the_plain_attention(cuda_device, d, hq):
    """A table of zeros leaves every output of the plain pass bit for bit, but dQ
    (whose adds have no fixed order: two runs of the plain pass differ as well)."""
    w = inputs.small(640, hq, 2, d, cp=2)
    x = inputs.make_inputs(w, device="cuda")
    t, buckets = torch.zeros((32, hq), device="cuda", dtype=torch.bfloat16), ops.log_buckets(32, 300)
    o, lse, o_res = ops.attn_fwd(w, x["q"], x["k"], x["v"])
    dq, dk, dv = ops.attn_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], o_res=o_res)
    got = _run(w, x, t, buckets)
    for a, b in ((o, got[0]), (lse, got[1]), (dk, got[3]), (dv, got[4])):
        assert torch.equal(a, b)
    assert (dq.float() - got[2].float()).abs().max() <= 2.0 ** -7 * dq.float().abs().max()


def test_softmax_scale_and_long_walk(cuda_device):
    """A scale of its own, through the descriptor, at a length whose walks pass
    every interval: against the oracle on one head."""
    w = inputs.small(1500, 1, 1, 64, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    buckets = ops.log_buckets(16, 1000)
    t = torch.randn((16, 1), device="cuda").to(torch.bfloat16)
    desc, bias = ops.make_desc(w, scale=0.3), buckets.struct(t)
    o, o_res, lse = torch.empty_like(x["q"]), torch.empty_like(x["q"]), torch.empty((1, 1, 1500), device="cuda")
    grads = [torch.empty_like(x[n]) for n in ("q", "k", "v")] + [torch.empty_like(t)]
    ws = [torch.empty(ops.loong_attn_bias_workspace_size(desc, bias, p), dtype=torch.uint8, device="cuda")
          for p in (0, 1)]
    ops.loong_attn_bias_fwd(desc, bias, x["q"], x["k"], x["v"], o, lse, o_res, ws[0])
    ops.loong_attn_bias_bwd(desc, bias, x["q"], x["k"], x["v"], o, o_res, lse, x["do"], *grads, ws[1])
    r = obias.forward_backward(to64(x["q"][0]), to64(x["k"][0]), to64(x["v"][0]), to64(x["do"][0]), to64(t),
                               buckets.bounds, buckets.bucket_of, 0.3, True, terms=True)
    e = _e(w, r)
    _within("O", o[0], r["o"], 2.0 ** -8 * np.abs(r["o"]) + (2.0 ** -11 + e + 2.0 ** -16) * r["abs_o"])
    f = 2.0 ** -11 + 2 * e + 2.0 ** -14
    for nm, got in zip(("dq", "dk", "dv"), grads):
        _within(nm, got[0], r[nm], 2.0 ** -8 * np.abs(r[nm]) + (2.0 ** -8 + f) * r["abs_" + nm])
    _within("dtable", grads[3], r["dtable"], 2.0 ** -8 * np.abs(r["dtable"]) + f * r["abs_dtable"])


def test_run_of_the_positional_operators(cuda_device):
    """A layer's attention as it is used: fused projection -> norm, rotation and
    the ranks' layout -> biased attention -> back to the projection's gradient,
    eagerly, on another stream, and captured and replayed on new inputs."""
    w = inputs.Workload("layer", 768, 4, 2, 64, 2, 3, 3, 1, True)
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    x = rn(1, 768, 8 * 64).to(torch.bfloat16)
    do = ops.headctx_pack(rn(1, 768, 4, 64).to(torch.bfloat16), w.cp, w.hp)
    wq, wk, t = 1 + 0.1 * rn(64), 1 + 0.1 * rn(64), rn(32, 4).to(torch.bfloat16)
    buckets, opts, lay = ops.log_buckets(32, 500), ops.make_qk_opts(64, base=500000.0), ops.LAYOUT_RANK_MAJOR
    split = lambda a: [u.unflatten(2, (-1, 64)) for u in a.split([256, 128, 128], dim=2)]

    def layer():
        dx = torch.empty_like(x)
        q, k, v = ops.qk_norm_rope(w, opts, *split(x), wq=wq, wk=wk, layout=lay)
        o, lse, res = ops.attn_bias_fwd(w, q, k, v, t, buckets, layout=lay)
        dq, dk, dv, dt = ops.attn_bias_bwd(w, q, k, v, o, lse, do, t, buckets, o_res=res, layout=lay)
        sq, sk, _ = split(x)
        _, _, _, dwq, dwk = ops.qk_norm_rope_bwd(w, opts, sq, sk, dq, dk, dv, wq=wq, wk=wk, layout=lay, into=split(dx))
        return o, lse, dt, dwk, dx, dwq

    def same(a, b):
        assert all(torch.equal(u, v) for u, v in zip(a[:4], b[:4]))
        for u, v in zip(a[4:], b[4:]):    # through dQ, whose fp32 adds have no fixed order before its bf16 rounding
            assert (u.float() - v.float()).abs().max() <= 2.0 ** -6 * v.float().abs().max()
    want = layer()
    # against the same layer in float64 torch, by its own differentiation
    from oracle import qk as oqk
    x64, ws64, t64 = x.double().requires_grad_(), [wq.double().requires_grad_(), wk.double().requires_grad_()], \
        t.double().requires_grad_()
    m = torch.from_numpy(oqk.matrices(range(768), 64, 64, oqk.frequencies(64, 500000.0), False, 1.0)).cuda()
    q, k, v = split(x64)
    q, k = (torch.einsum("tab,nthb->ntha", m, u * (u.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * wt)
            for u, wt in ((q, ws64[0]), (k, ws64[1])))
    n = torch.arange(768, device="cuda")[:, None] - torch.arange(768, device="cuda")
    ids = torch.from_numpy(obias.buckets_of_distance(n.cpu().numpy(), buckets.bounds, buckets.bucket_of)).cuda()
    logits = torch.einsum("nihd,njhd->nhij", q, k.repeat_interleave(2, 2)) / 8 + t64[ids].permute(2, 0, 1)
    p = logits.masked_fill(n < 0, -torch.inf).softmax(-1)
    o = torch.einsum("nhij,njhd->nihd", p, v.repeat_interleave(2, 2))
    grads = torch.autograd.grad(o, [x64, t64] + ws64, _unpack(w, do).double())
    # relative 2-norms: roundings to bf16 of Q, K, P, dS and the gradient (O: Q, K and O), of random sign, each at
    # most 2^-8, and the first two through an exponent: a logit of |q| |k| / 8 <= 8 sqrt 2 shifts by 8 * 2^-8 /
    # sqrt(64 / 2) or less in the mean square, under 2^-8 * sqrt 2
    far = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert far(_unpack(w, want[0]), o) < 5 ** 0.5 * 2.0 ** -8
    for got, ref in zip((want[4], want[2], want[5], want[3]), grads):
        assert far(got, ref) < 5 ** 0.5 * 2.0 ** -8
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer()
    s.synchronize()
    same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    x.copy_(rn(*x.shape).to(torch.bfloat16))
    t.copy_(rn(32, 4).to(torch.bfloat16))
    graph.replay()
    torch.cuda.synchronize()
    held = [u.clone() for u in held]
    same(held, layer())
    assert not torch.equal(held[0], want[0])
    assert ops.loong_get_device_status() == ops.LOONG_OK


@pytest.mark.parametrize("name", ["gqa", "not-causal", "empty-rows-ring", "group-of-34", "one-head-groups"])
def test_checked_build(cuda_device, monkeypatch, name):
    """The build with device address checks finds nothing to report."""
    monkeypatch.setattr(ops, "LIB_PATH", ops.CHECKED_LIB_PATH)
    monkeypatch.setattr(ops, "_lib", None)
    w, x, t, buckets = _make(name)
    _check(w, x, t, buckets, _run(w, x, t, buckets))


# S, hq, hkv, d, causal, buckets, the masked bucket: a window, a hole, many boundaries in a piece, both signs
MASKED = {
    "window": (900, 2, 1, 64, True, (3, [150, 400]), 2),
    "hole": (700, 4, 2, 128, True, (4, [3, 60, 333]), 1),
    "comb": (300, 2, 2, 64, True, (2, list(range(1, 200)), [i & 1 for i in range(200)]), 1),
    "band": (513, 2, 1, 128, False, (3, [-99, 100]), 0),
}


@pytest.mark.parametrize("value", [-30000.0, -65504.0, -1e9, -1e30])
@pytest.mark.parametrize("name", list(MASKED))
def test_finite_masks(cuda_device, name, value):
    """Masks written as large finite numbers: where every query keeps a key, exp(value) is 0 beside it in float64
    as well, so every output is that of -inf, within the tolerances of the other buckets' logits."""
    S, hq, hkv, d, causal, bk, at = MASKED[name]
    w = inputs.Workload(name, S, hq, hkv, d, 1, 1, 1, 1, True, placement=0, causal=causal)
    x, buckets = inputs.make_inputs(w, device="cuda"), ops.RelBuckets(*bk)
    t = torch.randn((buckets.num_buckets, hq), generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    t[at] = value
    t = t.to(torch.bfloat16)
    out = _run(w, x, t, buckets)
    t[at] = -torch.inf
    _check(w, x, t, buckets, out)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e9])
def test_buckets_out_of_reach(cuda_device, value):
    """What stands in buckets that no pair falls in (ahead of a causal query, beyond the sequence) changes no bit
    of what has a fixed order."""
    w = inputs.Workload("reach", 300, 4, 2, 64, 1, 3, 3, 1, True, placement=0)
    x, buckets = inputs.make_inputs(w, device="cuda"), ops.RelBuckets(5, [-40, 0, 33, 300])
    t = torch.randn((5, 4), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda").to(torch.bfloat16)
    t[0], t[1], t[4] = 0, 0, 0
    want = _run(w, x, t, buckets)
    t[0], t[1], t[4] = value, value, value
    got = _run(w, x, t, buckets)
    for i in (0, 1, 3, 4, 5):
        assert torch.equal(got[i], want[i])
    assert (got[2].float() - want[2].float()).abs().max() <= 2.0 ** -7 * want[2].float().abs().max()


@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 2.0 ** 20])
def test_values_out_of_range_show(cuda_device, value, mode):
    """Rows that meet one are NaN, the others as they were; so are the gradients of what those rows enter."""
    w = inputs.Workload("range", 400, 2, 1, 64, 1, 2, 2, 1, True, placement=0)
    x, buckets = inputs.make_inputs(w, device="cuda"), ops.RelBuckets(2, [170])
    t = torch.zeros((2, 2), device="cuda", dtype=torch.bfloat16)
    want = _run(w, x, t, buckets, mode=mode)
    t[1] = value
    o, lse, dq, dk, dv, dt = _run(w, x, t, buckets, mode=mode)
    assert torch.equal(o[:, :170], want[0][:, :170]) and torch.equal(lse[..., :170], want[1][..., :170])
    assert bool(o[:, 170:].isnan().all()) and bool(lse[..., 170:].isnan().all())
    for name, grad in (("dq", dq[:, 170:]), ("dk", dk), ("dv", dv), ("dtable", dt)):
        assert bool(grad.isnan().all()), name


@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE])
def test_plain_attention_shows_nan(cuda_device, mode):
    """Without a bias, a NaN key makes every row NaN that sees it."""
    w = inputs.Workload("nan", 400, 2, 1, 64, 1, 2, 2, 1, True, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    x["k"][:, 250, :, 3] = float("nan")
    o = ops.attn_fwd(w, x["q"], x["k"], x["v"], mode=mode)[0]
    assert bool(o[:, 250:].isnan().all()) and not bool(o[:, :250].isnan().any())


def test_long_context(cuda_device):
    """20,010 tokens on a ring of five: walks over many intervals, blocks that are no multiple of a tile, far
    boundaries.  Every output against float64 torch, rows of queries at a time, in the norm: each bf16 rounding
    (P, dS, the result) contributes at most 2^-8 / sqrt 3 of random sign, D 2^-11."""
    w = inputs.Workload("long", 20010, 2, 1, 64, 1, 5, 5, 1, True, placement=1)
    x = inputs.make_inputs(w, device="cuda")
    buckets = ops.RelBuckets(6, [1, 40, 1000, 5000, 15001])
    t = torch.randn((6, 2), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").to(torch.bfloat16)
    out = _run(w, x, t, buckets)
    q, k, v, do = (x[n][0].double() for n in ("q", "k", "v", "do"))
    S, scale = w.seqlen, 1 / 8
    want = [torch.zeros_like(q), torch.zeros((2, S), dtype=torch.float64, device="cuda"), torch.zeros_like(q),
            torch.zeros_like(k), torch.zeros_like(v), torch.zeros((6, 2), dtype=torch.float64, device="cuda")]
    bounds = torch.tensor(buckets.bounds, device="cuda")
    j = torch.arange(S, device="cuda")
    for i0 in range(0, S, 2048):
        i = torch.arange(i0, min(S, i0 + 2048), device="cuda")
        keys = int(i[-1]) + 1
        n = i[:, None] - j[:keys]
        ids = torch.bucketize(n, bounds, right=True)
        for h in range(2):
            logits = (scale * q[i, h] @ k[:keys, 0].T + t.double()[ids, h]).masked_fill(n < 0, -torch.inf)
            want[1][h, i] = torch.logsumexp(logits, -1)
            p = logits.softmax(-1)
            want[0][i, h] = p @ v[:keys, 0]
            ds = p * (do[i, h] @ v[:keys, 0].T - (do[i, h] * want[0][i, h]).sum(-1, keepdim=True))
            want[2][i, h] = scale * ds @ k[:keys, 0]
            want[3][:keys, 0] += scale * ds.T @ q[i, h]
            want[4][:keys, 0] += p.T @ do[i, h]
            want[5][:, h] += torch.bincount(ids.flatten(), ds.flatten(), minlength=6)
    far = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    assert far(out[1][0], want[1]) < 2.0 ** -20
    assert far(out[0][0], want[0]) < 2.0 ** -8
    for got, ref in zip((out[2][0], out[3][0], out[4][0], out[5]), want[2:]):
        assert far(got, ref) < 3 ** 0.5 * 2.0 ** -8


def test_two_calls_at_once(cuda_device):
    """Two streams at work together, each with workspaces of its own, give what they give alone."""
    cases = [_make(n) for n in ("ragged-blocks", "256-buckets")]
    alone = [_run(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[] for _ in cases]
    for _ in range(4):
        for i, (s, (w, x, t, buckets)) in enumerate(zip(streams, cases)):
            o, lse, res = ops.attn_bias_fwd(w, x["q"], x["k"], x["v"], t, buckets, stream=s)
            got[i].append((o, lse) + ops.attn_bias_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], t, buckets,
                                                       o_res=res, stream=s))
    torch.cuda.synchronize()
    for want, runs in zip(alone, got):
        for run in runs:
            for n, (a, b) in enumerate(zip(run, want)):
                if n == 2:    # dQ: its adds have no fixed order
                    assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * b.float().abs().max()
                else:
                    assert torch.equal(a, b)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,hq,hkv,copies", [(64, 2, 1, 1), (64, 3, 3, 1), (128, 2, 1, 1), (64, 3, 3, 20)])
def test_maxima_rise_on_every_tile(cuda_device, d, hq, hkv, copies, causal):
    """Keys whose scores rise by 8 from tile to tile, 11.5 in log2 units: every tile after the first rescales every
    row's accumulator, with one query tile per block (the few blocks) and with two (the copies).  The logits reach
    64, within what the tolerances count."""
    w = inputs.Workload("rise", 1100, hq, hkv, d, 1, 1, 1, 1, True, placement=0, causal=causal, batch=copies)
    x = inputs.make_inputs(w.with_(batch=1), device="cuda")
    x["q"][..., 0] = d ** 0.5
    x["k"][..., 0] = (8 * (torch.arange(1100, device="cuda") // 128)).to(torch.bfloat16)[None, :, None]
    x["q"][..., 1:] /= 8
    buckets = ops.log_buckets(16, 600, causal=causal)
    t = torch.randn((16, hq), generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").to(torch.bfloat16)
    out = _run(w, {n: v.repeat(copies, 1, 1, 1) for n, v in x.items()}, t, buckets)
    r = obias.forward_backward(to64(x["q"][0]), to64(x["k"][0]), to64(x["v"][0]), to64(x["do"][0]), to64(t),
                               buckets.bounds, buckets.bucket_of, ops.default_scale(d), causal, terms=True)
    e = _e(w, r)
    f = 2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -14
    for b in range(copies):
        _within("O", out[0][b], r["o"], 2.0 ** -8 * np.abs(r["o"]) + (2.0 ** -11 + e + 2.0 ** -16) * r["abs_o"])
        _within("LSE", out[1][b], r["lse"], e + 2.0 ** -22 * np.abs(r["lse"]))
        for nm, got in (("dq", out[2]), ("dk", out[3]), ("dv", out[4])):
            _within(nm, got[b], r[nm], 2.0 ** -8 * np.abs(r[nm]) + f * r["abs_" + nm])
    _within("dtable", out[5], copies * r["dtable"], copies * ((2.0 ** -11 + 2 * e + 2.0 ** -14) * r["abs_dtable"]
                                                               + 2.0 ** -8 * np.abs(r["dtable"])))


@pytest.mark.parametrize("mode", [ops.MODE_FUSED, ops.MODE_STEPWISE, ops.MODE_STEPWISE_COPY])
@pytest.mark.parametrize("d,hq,hkv,batch", [(64, 3, 1, 1), (64, 1, 1, 160), (128, 3, 1, 40), (128, 2, 2, 80)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 2.0 ** 20, -float("inf")])
def test_a_whole_tile_ahead_of_its_queries(cuda_device, value, d, hq, hkv, batch, mode):
    """The last head of an odd group pairs two of its query tiles, the first of which meets a key tile that lies
    ahead of all its queries, one interval for the whole of it: what stands there changes no bit."""
    w = inputs.Workload("ahead", 1068, hq, hkv, d, 1, 3, 3, 1, True, placement=0, batch=batch)
    x, buckets = inputs.make_inputs(w, device="cuda"), ops.RelBuckets(4, [0, 33, 300])
    t = torch.randn((4, hq), generator=torch.Generator(device="cuda").manual_seed(9), device="cuda").to(torch.bfloat16)
    lay = ops.LAYOUT_NATURAL
    if mode == ops.MODE_STEPWISE_COPY:
        x, lay = _pack(w, x), ops.LAYOUT_RANK_MAJOR
    t[0] = 0
    want = _run(w, x, t, buckets, mode=mode, layout=lay)
    t[0] = value
    got = _run(w, x, t, buckets, mode=mode, layout=lay)
    # in the stepwise modes dK and dV are summed by adds as well
    for i in (0, 1, 5) if mode != ops.MODE_FUSED else (0, 1, 3, 4, 5):
        assert torch.equal(got[i], want[i]), i
    for i in (2, 3, 4):
        assert (got[i].float() - want[i].float()).abs().max() <= 2.0 ** -7 * want[i].float().abs().max()
