"""Ring attention over key ranges with capped scores, and its gradients, against
the float64 oracle.

Tolerances, per element, from what rounds on the way (half steps: bf16 2^-8 of
the value, fp16 2^-11, fp32 2^-24):
  * a logit x: products of bf16 are exact, their sum takes at most d + 4 fp32
    roundings of at most L = scale |q| |k|max; the cap's tanh is off by at most
    2^-21 of the cap (and passes the score's own error on, its slope being at most
    1): dx = (d + 4) 2^-24 L + 2^-21 cap; the exponential and its argument 2^-21 +
    2^-23 L more: every P is off by at most a factor 1 + e, e = 2 (dx + 2^-21 +
    2^-23 L).
  * O: P rounded to fp16, sums in fp32, O to bf16: 2^-8 |O| + (2^-11 + e + 2^-16) A,
    A = P |V|; LSE: e + 2^-22 |LSE|.
  * the backward's P and dS are rounded to bf16, D comes from O and its residual
    (P to fp16: 2^-11 of A, then 2^-16): dS is off by at most
    f = 2^-8 + 2^-11 + 2 e + 2^-14 of a = P (|dO| |V| + |dO| A) times the cap's
    slope; the slope 1 - t^2 itself by at most 2 (2^-21) + 2^-23, dx / cap times 2
    more: g = 2^-19 + 2 dx / cap of a without it.  dQ, dK, dV by the same of their
    sums over absolute values, plus 2^-8 of themselves.
"""
import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import mask as omask
from tests.helpers import to64

pytestmark = pytest.mark.gpu


def _docs(*lengths, prefix=None, window=0, causal=True):
    return lambda w, g: ops.document_ranges([list(lengths)] * w.batch, w.seqlen, window=window, causal=causal,
                                            prefix=None if prefix is None else [list(prefix)] * w.batch)


def _random(w, g):
    """Every query its own range, many empty, some beyond both ends."""
    a = torch.randint(-20, w.seqlen + 20, (w.batch, w.seqlen), generator=g)
    n = torch.randint(-10, w.seqlen, (w.batch, w.seqlen), generator=g)
    return torch.stack((a, a + n), -1).to(torch.int32)


def _scattered(w, g):
    """Most queries see a few keys somewhere, tiles far apart."""
    a = torch.randint(0, w.seqlen, (w.batch, w.seqlen // 128 + 1, 1), generator=g).expand(-1, -1, 128)
    a = a.reshape(w.batch, -1)[:, :w.seqlen]
    return torch.stack((a, a + 3), -1).to(torch.int32)


def _nothing(w, g):
    return torch.full((w.batch, w.seqlen, 2), 7, dtype=torch.int32)


def _extreme(w, g):
    r = torch.empty((w.batch, w.seqlen, 2), dtype=torch.int32)
    r[..., 0], r[..., 1] = -2 ** 31, 2 ** 31 - 1
    r[:, 1::3] = torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    return r


# S, hq, hkv, d, hp, cp, inner, zigzag, batch, causal, cap, factor of q, ranges
CASES = {
    "one-token": (1, 2, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, _docs(1)),
    "one-token-padded": (1, 2, 2, 128, 1, 1, 1, 0, 2, 1, 5, 1, _docs()),
    "two-tokens": (2, 2, 2, 128, 1, 1, 1, 1, 3, 1, 5, 1, _docs(1, 1)),
    "three-keys": (3, 2, 1, 64, 1, 3, 3, 0, 1, 0, 0, 1, _docs(2, causal=False)),
    "under-a-tile": (100, 4, 2, 64, 1, 1, 1, 0, 1, 1, 30, 3, _docs(30, 1, 50)),
    "tile-and-one": (129, 3, 1, 128, 1, 1, 1, 0, 1, 1, 0, 1, _docs(127, 2)),
    "gqa": (512, 4, 2, 64, 2, 4, 2, 1, 1, 1, 0, 1, _docs(100, 200, 212)),
    "ragged-blocks": (600, 2, 1, 128, 1, 3, 3, 1, 1, 1, 50, 3, _docs(250, 300, 7)),
    "whole": (398, 2, 2, 64, 1, 2, 2, 0, 2, 0, 20, 1, _docs(130, 200, causal=False)),
    "whole-window": (500, 2, 2, 64, 1, 2, 2, 0, 1, 0, 0, 1, _docs(300, 200, causal=False, window=40)),
    "prefix": (700, 2, 1, 128, 1, 2, 1, 1, 1, 0, 0, 1, _docs(300, 350, prefix=(170, 400))),
    "window": (900, 2, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, _docs(900, window=150)),
    "window-one": (300, 2, 1, 128, 1, 1, 1, 0, 1, 1, 0, 1, _docs(300, window=1)),
    "many-documents": (640, 2, 1, 128, 1, 1, 1, 0, 1, 1, 0, 1, _docs(*[20] * 32)),
    "tile-documents": (1024, 2, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, _docs(*[128] * 8)),
    "padding": (1000, 2, 2, 64, 1, 1, 1, 0, 2, 1, 0, 1, _docs(100, 150)),
    "padding-first-doc-empty": (260, 2, 2, 64, 1, 1, 1, 0, 1, 1, 0, 1, _docs(0, 3, 0)),
    "random": (700, 3, 1, 64, 1, 1, 1, 0, 2, 0, 0, 1, _random),
    "random-causal-ring": (768, 4, 2, 128, 2, 3, 3, 1, 1, 1, 15, 3, _random),
    "scattered": (1500, 2, 1, 64, 1, 1, 1, 0, 1, 0, 0, 1, _scattered),
    "nothing": (300, 2, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, _nothing),
    "extreme-ranges": (300, 2, 1, 128, 1, 1, 1, 0, 1, 0, 0, 1, _extreme),
    "cap-alone": (500, 4, 2, 64, 1, 1, 1, 0, 1, 1, 30, 1, None),
    "cap-alone-whole": (333, 2, 2, 128, 1, 1, 1, 0, 2, 0, 10, 2, None),
    "cap-saturated": (400, 2, 1, 64, 1, 1, 1, 0, 1, 1, 2, 40, None),
    "cap-small": (400, 2, 1, 128, 1, 1, 1, 0, 1, 1, 2.0 ** -20, 1, None),
    "cap-large": (400, 2, 1, 128, 1, 1, 1, 0, 1, 1, 2.0 ** 20, 1, None),
    "neither": (300, 2, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, None),
    "one-head-groups": (600, 3, 3, 128, 1, 1, 1, 0, 1, 1, 0, 1, _docs(200, 400)),
    "one-head-tile-pairs": (1300, 2, 2, 64, 1, 2, 2, 1, 8, 0, 0, 1, _docs(100, 30, 600, causal=False)),
    "groups-of-five": (420, 10, 2, 64, 1, 1, 1, 0, 1, 1, 30, 3, _docs(170, 250)),
    "group-of-34": (150, 34, 1, 64, 1, 1, 1, 0, 1, 1, 0, 1, _docs(70, 60)),
    "flushes": (4200, 16, 1, 64, 1, 1, 1, 0, 1, 0, 0, 1, _docs(4200, causal=False)),
}


def _make(name, seed=0):
    S, hq, hkv, d, hp, cp, inner, zz, B, causal, cap, mul, ranges = CASES[name]
    w = inputs.Workload(name, S, hq, hkv, d, hp, cp, inner, cp // inner, True, placement=zz, batch=B,
                        causal=bool(causal))
    x = inputs.make_inputs(w, device="cuda", seed_offset=seed)
    x["q"] = (x["q"].float() * mul).to(torch.bfloat16)
    r = None if ranges is None else ranges(w, torch.Generator().manual_seed(7 + seed))
    return w, x, r, float(cap)


def _pack(w, x):
    return {n: ops.headctx_pack(t, w.cp, w.hp, 1 if w.placement else 2) for n, t in x.items()}


def _unpack(w, t):
    return ops.headctx_unpack(t, w.batch, w.cp, w.hp, 1 if w.placement else 2)


def _run(w, x, r, cap, mode=ops.MODE_FUSED, layout=ops.LAYOUT_NATURAL, res=True):
    r = None if r is None else r.cuda()
    o, lse, o_res = ops.attn_mask_fwd(w, x["q"], x["k"], x["v"], r, cap, mode=mode, layout=layout, res=res)
    grads = ops.attn_mask_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], r, cap, o_res=o_res, mode=mode,
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


def _sees(w, r, b):
    rb = np.tile([0, w.seqlen], (w.seqlen, 1)) if r is None else r[b].numpy()
    return omask.sees(rb, w.seqlen, w.causal)


def _check(w, x, r, cap, out):
    o, lse, dq, dk, dv = out
    for b in range(w.batch):
        t = omask.forward_backward(to64(x["q"][b]), to64(x["k"][b]), to64(x["v"][b]), to64(x["do"][b]),
                                   _sees(w, r, b), ops.default_scale(w.head_dim), cap, terms=True)
        L = t["logit"].max()
        dx = (w.head_dim + 4) * 2.0 ** -24 * L + 2.0 ** -21 * cap
        e = 2 * (dx + 2.0 ** -21 + 2.0 ** -23 * (min(L, cap) if cap else L))
        _within("O", o[b], t["o"], 2.0 ** -8 * np.abs(t["o"]) + (2.0 ** -11 + e + 2.0 ** -16) * t["abs_o"])
        some = np.isfinite(t["lse"])
        _within("LSE", lse[b], t["lse"], np.where(some, e + 2.0 ** -22 * np.abs(np.where(some, t["lse"], 0)), 0))
        f = 2.0 ** -8 + 2.0 ** -11 + 2 * e + 2.0 ** -14
        g = 2.0 ** -19 + 2 * dx / cap if cap else 0.0
        for nm, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            _within(nm, got[b], t[nm], 2.0 ** -8 * np.abs(t[nm]) + f * t["abs_" + nm] + g * t["flat_" + nm])


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(cuda_device, name):
    w, x, r, cap = _make(name)
    _check(w, x, r, cap, _run(w, x, r, cap))


@pytest.mark.parametrize("name", ["gqa", "ragged-blocks", "whole", "prefix", "random-causal-ring", "three-keys",
                                  "one-head-tile-pairs", "two-tokens"])
@pytest.mark.parametrize("mode", [ops.MODE_STEPWISE, ops.MODE_STEPWISE_COPY, ops.MODE_STEPWISE_COPY_AB])
def test_stepwise(cuda_device, name, mode):
    w, x, r, cap = _make(name)
    if mode == ops.MODE_STEPWISE:
        _check(w, x, r, cap, _run(w, x, r, cap, mode=mode))
        return
    if mode == ops.MODE_STEPWISE_COPY_AB and not w.placement:
        w = w.with_(placement=1)
        if w.seqlen % (2 * w.cp * w.hp):
            pytest.skip("the length does not divide into paired blocks")
    out = _run(w, _pack(w, x), r, cap, mode=mode, layout=ops.LAYOUT_RANK_MAJOR)
    _check(w, x, r, cap, [t if i == 1 else _unpack(w, t) for i, t in enumerate(out)])


@pytest.mark.parametrize("name", ["gqa", "ragged-blocks", "prefix", "random-causal-ring", "one-head-tile-pairs"])
def test_rank_major(cuda_device, name):
    w, x, r, cap = _make(name)
    out = _run(w, _pack(w, x), r, cap, layout=ops.LAYOUT_RANK_MAJOR)
    _check(w, x, r, cap, [t if i == 1 else _unpack(w, t) for i, t in enumerate(out)])


def test_causal_ranges_equal_plain(cuda_device):
    """Ranges that leave everything: the causal forward's values to its rounding."""
    w = inputs.small(1024, 4, 2, 128, 2, 2)
    x = inputs.make_inputs(w, device="cuda")
    o, lse, _ = ops.attn_fwd(w, x["q"], x["k"], x["v"])
    o2, lse2, _ = ops.attn_mask_fwd(w, x["q"], x["k"], x["v"])
    assert (o.float() - o2.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert (lse - lse2).abs().max() <= 2.0 ** -18


def _poisoned(x, names, where, value):
    y = {n: t.clone() for n, t in x.items()}
    for n in names:
        y[n][where] = value
    return y


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seqlen,cp,docs,cap", [(300, 1, (100, 120), 0.0), (398, 1, (150, 90), 20.0),
                                                (398, 2, (140, 90), 0.0)])
def test_padding_holds_anything(cuda_device, value, d, seqlen, cp, docs, cap):
    """Tokens behind the last document may hold anything: outputs and gradients of the others are the same bits (dQ,
    which is added up in any order, to rounding), their own are 0."""
    w = inputs.Workload("pad", seqlen, 4, 2, d, 1, cp, cp, 1, True, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    x["q"] = x["q"] * 8  # with the cap, in reach of every form of it
    r = ops.document_ranges([list(docs)], seqlen)
    end = sum(docs)
    clean = _run(w, x, r, cap)
    y = _poisoned(x, ("q", "k", "v", "do"), (slice(None), slice(end, None)), value)
    got = _run(w, y, r, cap)
    _check(w, x, r, cap, got)
    for i, (a, b) in enumerate(zip(clean, got)):
        if i != 2:
            assert torch.equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else torch.int32),
                               b.view(torch.int16 if b.dtype == torch.bfloat16 else torch.int32)), i


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_other_documents_hold_anything(cuda_device, value, name, cap):
    """A value that is not finite stays within its document, whose ends lie inside tiles."""
    w = inputs.Workload("docs", 500, 4, 2, 64, 1, 1, 1, 1, True, placement=0)
    x = inputs.make_inputs(w, device="cuda")
    r = ops.document_ranges([[130, 170, 200]], 500)
    at = 140 if name in ("k", "v") else 290
    y = _poisoned(x, (name,), (0, at, 0, 5), value)
    with_do = dict(y)
    o, lse, dq, dk, dv = _run(w, with_do, r, cap)
    out = [o, lse, dq, dk, dv]
    keep = [i for i in range(500) if i < 130 or i >= 300]
    t = omask.forward_backward(to64(x["q"][0]), to64(x["k"][0]), to64(x["v"][0]), to64(x["do"][0]), _sees(w, r, 0),
                               ops.default_scale(64), cap)
    for nm, got in zip(("o", "lse", "dq", "dk", "dv"), out):
        got, want = to64(got[0]), t[nm]
        if nm == "lse":
            got, want = got.T, want.T
        near = np.abs(got[keep] - want[keep]) <= 0.05 * (1 + np.abs(want[keep]))
        assert near.all(), f"{nm}: {near.size - near.sum()} of {near.size} values of other documents changed"
    # a finite cap makes a finite score of an infinite one; everything else shows
    if not (cap and value == float("inf") and name in ("q", "k")):
        seen = {"q": ("o", "lse", "dq", "dk", "dv"), "k": ("o", "lse", "dq"), "v": ("o", "dq"), "do": ("dk", "dv", "dq")}
        heads = {"q": 0, "do": 0, "k": slice(0, 2), "v": slice(0, 2)}[name]
        for nm, got in zip(("o", "lse", "dq", "dk", "dv"), out):
            if nm not in seen[name]:
                continue
            g = to64(got[0])
            g = g.T[..., None] if nm == "lse" else g
            if nm in ("dk", "dv"):
                assert not np.isfinite(g[150:285, 0]).all(), nm
            else:
                rows = g[290, heads] if name in ("q", "do") else g[140:300, heads]
                assert not np.isfinite(rows).any(axis=-1).all(), nm


def test_gradients_by_differences(cuda_device):
    """The gradient of sum(O dO) against central differences of the oracle's forward in 64 bits."""
    w, x, r, cap = _make("under-a-tile")
    dq, dk, dv = _run(w, x, r, cap)[2:]
    see, scale = _sees(w, r, 0), ops.default_scale(w.head_dim)
    base = {n: to64(t[0]) for n, t in x.items()}
    rng = np.random.default_rng(0)
    for nm, got in (("q", dq), ("k", dk), ("v", dv)):
        step = rng.standard_normal(base[nm].shape)
        f = []
        for sign in (1, -1):
            y = dict(base)
            y[nm] = base[nm] + sign * 1e-4 * step
            f.append((omask.forward_backward(y["q"], y["k"], y["v"], None, see, scale, cap)["o"] * base["do"]).sum())
        want = (f[0] - f[1]) / 2e-4
        g = to64(got[0])
        assert abs((g * step).sum() - want) <= 2.0 ** -7 * np.linalg.norm(g) * np.linalg.norm(step) ** 0.5 + 1e-3


def test_graph_and_streams(cuda_device):
    """A training step captured into a graph and replayed on new inputs, the ranges' contents among them, beside the
    same step on another stream."""
    w, x, r, cap = _make("under-a-tile")
    w2, x2, r2, _ = _make("under-a-tile", seed=3)
    r2 = ops.document_ranges([[7, 60, 20]], w.seqlen)
    buf = {n: t.clone() for n, t in x.items()}
    rb = r.cuda()

    def step(z, ranges):
        o, lse, o_res = ops.attn_mask_fwd(w, z["q"], z["k"], z["v"], ranges, cap)
        return (o, lse) + ops.attn_mask_bwd(w, z["q"], z["k"], z["v"], o, lse, z["do"], ranges, cap, o_res=o_res)
    step(buf, rb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(buf, rb)
    for z, ranges in ((x2, r2), (x, r)):
        for n in buf:
            buf[n].copy_(z[n])
        rb.copy_(ranges)
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = step(x2, r2.cuda())
        torch.cuda.synchronize()
        _check(w, z, ranges, cap, out)
        _check(w, x2, r2, cap, other)
    assert ops.loong_get_device_status() == ops.LOONG_OK


def test_stream_argument(cuda_device):
    w, x, r, cap = _make("gqa")
    rc = r.cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        o, lse, res = ops.attn_mask_fwd(w, x["q"], x["k"], x["v"], rc, cap, stream=stream)
        g = ops.attn_mask_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], rc, cap, o_res=res, stream=stream)
        s.synchronize()
        _check(w, x, r, cap, (o, lse) + g)


def test_without_residual(cuda_device):
    w, x, r, cap = _make("gqa")
    o, lse, dq, dk, dv = _run(w, x, r, cap, res=False)
    t = omask.forward_backward(to64(x["q"][0]), to64(x["k"][0]), to64(x["v"][0]), to64(x["do"][0]), _sees(w, r, 0),
                               ops.default_scale(w.head_dim), cap, terms=True)
    for nm, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        # D from O rounded to bf16: 2^-8 of |dO| |O| more
        _within(nm, got[0], t[nm], 2.0 ** -8 * np.abs(t[nm]) + 2.0 ** -6 * t["flat_" + nm])


def test_refusals(cuda_device):
    w, x, r, cap = _make("gqa")
    rc = r.cuda()
    q, k, v = x["q"], x["k"], x["v"]
    with pytest.raises(ValueError, match="key_range"):
        ops.attn_mask_fwd(w, q, k, v, rc.long())
    with pytest.raises(ValueError, match="key_range"):
        ops.attn_mask_fwd(w, q, k, v, rc[:, :-1])
    with pytest.raises(ValueError, match="key_range"):
        ops.attn_mask_fwd(w, q, k, v, r)
    with pytest.raises(ValueError, match="key_range must be contiguous"):
        ops.attn_mask_fwd(w, q, k, v, rc.expand(1, -1, -1).flip(2).transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="q must be"):
        ops.attn_mask_fwd(w, q.float(), k, v, rc)
    with pytest.raises(ops.LoongError):
        ops.attn_mask_fwd(w, q, k, v, rc, -1.0)
    desc, mask = ops.make_desc(w), ops.make_mask(rc, cap)
    n = ops.loong_attn_mask_workspace_size(desc, mask, 0)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((1, w.hq, w.seqlen), device="cuda")
    with pytest.raises(ops.LoongError) as err:
        ops.loong_attn_mask_fwd(desc, mask, q, k, v, o, lse, None, ws[:-16])
    assert err.value.status == ops.LOONG_ERR_WORKSPACE
    mask.key_range = r.data_ptr()  # host memory
    with pytest.raises(ops.LoongError) as err:
        ops.loong_attn_mask_fwd(desc, mask, q, k, v, o, lse, None, ws)
    assert err.value.status == ops.LOONG_ERR_INVALID_ARG
    mask.key_range = rc.data_ptr() + 4
    with pytest.raises(ops.LoongError) as err:
        ops.loong_attn_mask_fwd(desc, mask, q, k, v, o, lse, None, ws)
    assert err.value.status == ops.LOONG_ERR_INVALID_ARG
