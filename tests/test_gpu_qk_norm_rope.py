"""qk_norm_rope and its gradient against the float64 oracle.

Tolerances, per element, in units of what the value is made of (u = 2^-24, half
a step of fp32 1.0):
  * forward: one rounding to bf16, 2^-8 |y|; before it, at most 12 roundings in
    the sum of squares, 2 u each in rsqrt and the products, and an error of the
    angle's cosine and sine of 2^-24 (fraction of a turn) * 2 pi plus sincospi's
    2 u: together below 32 u = 2^-19 of |a| + |b|, the rotated pair's magnitudes
    (of the normed elements, times rot_scale).
  * dx: the same with h = g w and x r mean(h x r): 2^-8 |dx| + 2^-18 r (|h| +
    |x r| mean |h x r|), |h| from the pair's magnitudes.
  * dw: sums in chains of at most the heads of a token and the tokens of a warp
    (together under 256 here), then of 16 lanes per warp: under 2^-15 of the sum
    of |g x r|.
"""
import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import qk as oqk
from tests.helpers import to64

pytestmark = pytest.mark.gpu

# B, S, hq, hkv, d, hp, cp, zigzag, rank-major, rot, interleaved, fused projection, positions, norm, weights, rot_scale
CASES = {
    "one-token": (1, 1, 4, 2, 128, 1, 1, 0, 0, 128, 0, 1, "begin", 1, 1, 1.0),
    "one-token-b5": (5, 1, 3, 1, 64, 1, 1, 0, 0, 64, 0, 1, "any", 1, 1, 1.0),
    "one-token-b300": (300, 1, 8, 8, 64, 1, 1, 0, 0, 64, 1, 0, "any", 1, 1, 1.0),
    "two-tokens": (1, 2, 1, 1, 64, 1, 1, 1, 0, 64, 0, 0, None, 1, 1, 1.0),
    "odd": (3, 101, 5, 5, 128, 1, 1, 0, 0, 128, 0, 1, "any", 1, 1, 1.0),
    "odd-heads-d64": (2, 77, 7, 1, 64, 1, 1, 0, 0, 64, 0, 1, None, 1, 1, 1.0),
    "part-16": (1, 50, 6, 2, 128, 1, 1, 0, 0, 16, 0, 1, "any", 1, 1, 1.0),
    "part-96": (1, 50, 6, 2, 128, 1, 1, 0, 0, 96, 0, 1, "any", 1, 1, 1.0),
    "part-48-inter": (2, 33, 6, 2, 64, 1, 1, 0, 0, 48, 1, 1, "any", 1, 1, 1.0),
    "inter-128": (1, 40, 4, 4, 128, 1, 1, 0, 0, 128, 1, 0, None, 1, 1, 1.0),
    "no-rotation": (1, 40, 4, 4, 128, 1, 1, 0, 0, 0, 0, 1, None, 1, 1, 1.0),
    "no-norm": (2, 40, 4, 2, 128, 1, 1, 0, 0, 128, 0, 1, "any", 0, 0, 1.5),
    "neither": (1, 48, 4, 2, 64, 2, 3, 1, 1, 0, 0, 1, None, 0, 0, 1.0),
    "no-weights": (1, 40, 4, 2, 64, 1, 1, 0, 0, 64, 1, 0, None, 1, 0, 0.75),
    "ranks-zigzag": (1, 96, 8, 4, 128, 4, 3, 1, 1, 128, 0, 1, None, 1, 1, 1.0),
    "ranks-contiguous": (2, 90, 6, 3, 64, 3, 5, 0, 1, 32, 1, 1, "any", 1, 1, 1.0),
    "natural-mesh": (1, 96, 8, 4, 128, 4, 3, 1, 0, 128, 0, 1, None, 1, 1, 1.0),
    "many-heads": (1, 3, 99, 33, 64, 1, 1, 0, 0, 64, 0, 1, None, 1, 1, 1.0),
}
EPS, W_OFFSET = 1e-3, 0.25


def _make(name, seed=0):
    B, S, hq, hkv, d, hp, cp, zz, rm, rot, inter, fused, pos, norm, weights, rs = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(seed + S + d + hq)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")
    w = inputs.Workload(name, S, hq, hkv, d, hp, cp, cp, 1, True, batch=B, placement=zz)
    x = (rn(B, S, (hq + 2 * hkv) * d) * 2).to(torch.bfloat16)
    q, k, v = [t.unflatten(2, (-1, d)) for t in x.split([hq * d, hkv * d, hkv * d], dim=2)]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    c = dict(w=w, q=q, k=k, v=v, layout=ops.LAYOUT_RANK_MAJOR if rm else ops.LAYOUT_NATURAL,
             wq=1 + 0.3 * rn(d) if weights else None, wk=1 + 0.3 * rn(d) if weights else None, pos_begin=0,
             positions=None, fused=fused, norm=bool(norm), x=x)
    if pos == "begin":
        c["pos_begin"] = 777
    if pos == "any":
        c["positions"] = torch.randint(-1000, 1 << 20, (B, S), generator=g, device="cuda")
    c["opts"] = ops.make_qk_opts(d, eps=EPS, norm=bool(norm), w_offset=W_OFFSET, rot_dim=rot, base=10000.0,
                                 interleaved=bool(inter), rot_scale=rs)
    c["grads"] = [rn(B, S, h, d).to(torch.bfloat16) for h in (hq, hkv, hkv)]
    c["rot"] = (rot, bool(inter), rs)
    return c


def _lay(c, t):
    """[B, S, H, d] -> the case's layout, by the repack the suite checks on its own."""
    if c["layout"] == ops.LAYOUT_NATURAL:
        return t.contiguous()
    w = c["w"]
    return ops.headctx_pack(t.contiguous(), w.cp, w.hp, 1 if w.placement else 2)


def _lay64(c, a):
    """The case's layout of a float64 array (an index map of whole elements)."""
    t = torch.from_numpy(np.ascontiguousarray(a))
    if c["layout"] == ops.LAYOUT_NATURAL:
        return a
    w = c["w"]
    n = 2 * w.cp if w.placement else w.cp
    blk = w.seqlen // n
    order = [t0 for r in range(w.cp) for bl in ((r, n - 1 - r) if w.placement else (r,))
             for t0 in range(bl * blk, (bl + 1) * blk)]
    y = t[:, order].reshape(w.batch * w.cp, w.seqlen // w.cp, w.hp, -1, w.head_dim)
    return y.transpose(1, 2).numpy()


def _matrices(c, b):
    rot, inter, rs = c["rot"]
    S, d = c["w"].seqlen, c["w"].head_dim
    pos = c["pos_begin"] + np.arange(S) if c["positions"] is None else c["positions"][b].cpu().numpy()
    return oqk.matrices(pos, d, rot, oqk.frequencies(rot, 10000.0) if rot else [], inter, rs)


def _magnitude(c, m):
    """Ones where a pair's elements meet, times rot_scale."""
    return np.where(m != 0, max(1.0, c["rot"][2]), 0.0)


def _check(name, got, want, tol):
    got = to64(got)
    assert got.shape == want.shape and np.all(np.isfinite(got)), name
    err = np.abs(got - want)
    assert np.all(err <= tol), \
        f"{name}: {(err > tol).sum()} of {err.size} outside, worst {np.max(err / (tol + 1e-300)):.3g} of the tolerance"


def _place(c):
    return dict(wq=c["wq"], wk=c["wk"], positions=c["positions"], pos_begin=c["pos_begin"], layout=c["layout"])


@pytest.mark.parametrize("name", list(CASES))
def test_forward_matches_oracle(cuda_device, name):
    c = _make(name)
    got = ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], **_place(c))
    assert ops.loong_get_device_status() == ops.LOONG_OK
    assert torch.equal(got[2].view(torch.int16), _lay(c, c["v"]).view(torch.int16))
    for x, w, y in ((c["q"], c["wq"], got[0]), (c["k"], c["wk"], got[1])):
        want, tol = np.zeros(x.shape), np.zeros(x.shape)
        for b in range(x.shape[0]):
            m = _matrices(c, b)
            x64, w64 = to64(x[b]), None if w is None else to64(w)
            want[b] = oqk.forward(x64, w64, m, EPS, c["norm"], W_OFFSET)
            n = oqk.forward(x64, w64, np.broadcast_to(np.eye(x.shape[-1]), m.shape), EPS, c["norm"], W_OFFSET)
            tol[b] = 2.0 ** -8 * np.abs(want[b]) + 2.0 ** -19 * np.einsum("tab,thb->tha", _magnitude(c, m), np.abs(n))
        _check("y", y, _lay64(c, want), _lay64(c, tol))


@pytest.mark.parametrize("name", list(CASES))
def test_backward_matches_oracle(cuda_device, name):
    c = _make(name)
    into, dx = None, None
    if c["fused"]:
        dx = torch.full_like(c["x"], 7.0)
        w = c["w"]
        into = [t.unflatten(2, (-1, w.head_dim)) for t in dx.split(
            [w.hq * w.head_dim, w.hkv * w.head_dim, w.hkv * w.head_dim], dim=2)]
    dy = [_lay(c, g) for g in c["grads"]]
    run = lambda: ops.qk_norm_rope_bwd(c["w"], c["opts"], c["q"], c["k"], *dy, into=into, **_place(c))
    dq, dk, dv, dwq, dwk = run()
    assert ops.loong_get_device_status() == ops.LOONG_OK
    assert torch.equal(dv.contiguous().view(torch.int16), c["grads"][2].view(torch.int16))
    for x, w, g, dx_, dw in ((c["q"], c["wq"], c["grads"][0], dq, dwq), (c["k"], c["wk"], c["grads"][1], dk, dwk)):
        assert (dw is None) == (w is None or not c["norm"])
        want, tol = np.zeros(x.shape), np.zeros(x.shape)
        want_w, tol_w = 0, 0
        for b in range(x.shape[0]):
            m = _matrices(c, b)
            x64, w64 = to64(x[b]), None if w is None else to64(w)
            want[b], dwb = oqk.backward(x64, w64, m, EPS, to64(g[b]), c["norm"], W_OFFSET)
            gm = np.einsum("tba,thb->tha", _magnitude(c, m), np.abs(to64(g[b])))
            if c["norm"]:
                r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + EPS)
                h = gm * (1.0 if w is None else np.abs(w64 + W_OFFSET))
                xr = np.abs(x64 * r)
                tol[b] = 2.0 ** -18 * r * (h + xr * (h * xr).mean(-1, keepdims=True))
                want_w, tol_w = want_w + dwb, tol_w + 2.0 ** -15 * (gm * xr).sum((0, 1))
            else:
                tol[b] = 2.0 ** -18 * gm
        _check("dx", dx_, want, tol + 2.0 ** -8 * np.abs(want))
        if dw is not None:
            _check("dw", dw, want_w, tol_w)
    # the same bits again
    keep = [t.clone() for t in (dq, dk, dv)] + [dwq, dwk]
    for a, b in zip(keep, run()):
        assert (a is None and b is None) or torch.equal(a, b)


def test_far_positions(cuda_device):
    """Angles of positions near 2^31: the table's 2^-53 times the position is
    2^-22 of a radian, the fp32 steps as above; a reduction in fp32 would be off
    by whole turns."""
    w = inputs.small(4, 1, 1, 64, placement=0)
    q = torch.randn((1, 4, 1, 64), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 2 ** 30 + 1]], device="cuda")
    opts = ops.make_qk_opts(64, norm=False)
    y, _, _ = ops.qk_norm_rope(w, opts, q, q, positions=pos)
    m = oqk.matrices(pos[0].tolist(), 64, 64, oqk.frequencies(64, 10000.0), False, 1.0)
    want = oqk.forward(to64(q[0]), None, m, 0, norm=False)
    mag = np.einsum("tab,thb->tha", np.where(m != 0, 1.0, 0.0), np.abs(to64(q[0])))
    # four roundings of the table and the oracle's angle (2^31 * 2^-53 each) and 2^-19
    _check("y", y[0], want, 2.0 ** -8 * np.abs(want) + (2.0 ** -19 + 4 * 2.0 ** -22) * mag)


def test_given_frequencies_equal_the_base(cuda_device):
    c = _make("odd")
    a = ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], **_place(c))
    same = ops.make_qk_opts(128, eps=EPS, w_offset=W_OFFSET, inv_freq=oqk.frequencies(128, 10000.0))
    b = ops.qk_norm_rope(c["w"], same, c["q"], c["k"], c["v"], **_place(c))
    # Python's and C's pow may differ in the last bit of a frequency, 2^-53 of the angle: far below bf16
    for x, y in zip(a, b):
        assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * x.float().abs().max()


def test_v_left_out_and_gaps_left_alone(cuda_device):
    """Without v nothing of v is written; a strided gradient leaves the elements
    between a token's heads and the next token as they were."""
    w = inputs.small(37, 3, 3, 64, placement=0)
    wide = torch.randn((1, 37, 3 * 3 * 64 + 40), device="cuda").to(torch.bfloat16)
    q, k = (wide[:, :, i * 192:(i + 1) * 192].unflatten(2, (3, 64)) for i in (0, 1))
    opts = ops.make_qk_opts(64)
    qo, ko, vo = ops.qk_norm_rope(w, opts, q, k)
    assert vo is None
    dwide = torch.full_like(wide, 3.0)
    into = [dwide[:, :, i * 192:(i + 1) * 192].unflatten(2, (3, 64)) for i in (0, 1)] + [None]
    out = ops.qk_norm_rope_bwd(w, opts, q, k, qo, ko, into=into)
    assert out[2:] == (None, None, None)
    assert torch.all(dwide[:, :, 384:] == 3.0)
    ref = ops.qk_norm_rope_bwd(w, opts, q, k, qo, ko)
    assert torch.equal(ref[0], into[0]) and torch.equal(ref[1], into[1])


def test_zero_head_and_large_values(cuda_device):
    """A head of zeros has r = 1 / sqrt(eps) and stays 0, with dx = r h; values
    near 2^60 norm to the same as near 1."""
    w = inputs.small(2, 2, 2, 128, placement=0)
    opts = ops.make_qk_opts(128, eps=1e-4, rot_dim=0)
    q = torch.zeros((1, 2, 2, 128), device="cuda", dtype=torch.bfloat16)
    q[0, 1] = torch.randn((2, 128), device="cuda").to(torch.bfloat16)
    y, big, _ = ops.qk_norm_rope(w, opts, q, q * 2.0 ** 60)
    assert torch.all(y[0, 0] == 0) and torch.all(big[0, 0] == 0)
    # eps = 1e-4 against a mean square near 1: r differs by 5e-5 relative, below half a bf16 step
    assert (y.float() - big.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()
    g = torch.randn((1, 2, 2, 128), device="cuda").to(torch.bfloat16)
    dq, _, _, _, _ = ops.qk_norm_rope_bwd(w, opts, q, q, g, g)
    assert torch.allclose(dq[0, 0].float(), g[0, 0].float() * 100, rtol=2.0 ** -7, atol=0)


@pytest.mark.parametrize("name", ["odd", "odd-heads-d64", "part-48-inter"])
def test_eps_zero(cuda_device, name):
    """Without eps, heads that do not fill a warp: the lanes past the last head add nothing to dw."""
    c = _make(name)
    opts = ops.make_qk_opts(c["w"].head_dim, eps=0.0, w_offset=W_OFFSET, rot_dim=c["rot"][0], base=10000.0,
                            interleaved=c["rot"][1])
    out = ops.qk_norm_rope_bwd(c["w"], opts, c["q"], c["k"], *[_lay(c, g) for g in c["grads"]], **_place(c))
    for x, w, g, dx, dw in ((c["q"], c["wq"], c["grads"][0], out[0], out[3]),
                            (c["k"], c["wk"], c["grads"][1], out[1], out[4])):
        want_w, tol_w = 0, 0
        for b in range(x.shape[0]):
            m, x64 = _matrices(c, b), to64(x[b])
            want, dwb = oqk.backward(x64, to64(w), m, 0.0, to64(g[b]), True, W_OFFSET)
            gm = np.einsum("tba,thb->tha", _magnitude(c, m), np.abs(to64(g[b])))
            r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True))
            h, xr = gm * np.abs(to64(w) + W_OFFSET), np.abs(x64 * r)
            _check("dx", dx[b], want,
                   2.0 ** -8 * np.abs(want) + 2.0 ** -18 * r * (h + xr * (h * xr).mean(-1, keepdims=True)))
            want_w, tol_w = want_w + dwb, tol_w + 2.0 ** -15 * (gm * xr).sum((0, 1))
        _check("dw", dw, want_w, tol_w)


def test_other_stream_and_graph(cuda_device):
    """On a stream of its own, and captured once and replayed on new inputs: the
    bits of the eager calls on the default stream."""
    c = _make("ranks-zigzag")
    dy = [_lay(c, g) for g in c["grads"]]

    def run():
        y = ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], **_place(c))
        return y + ops.qk_norm_rope_bwd(c["w"], c["opts"], c["q"], c["k"], *dy, **_place(c))
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    other = _make("ranks-zigzag", seed=9)
    c["x"].copy_(other["x"])
    for a, b in zip(dy, other["grads"]):
        a.copy_(_lay(c, b))
    graph.replay()
    torch.cuda.synchronize()
    held = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(run(), held))
    assert not torch.equal(held[0], want[0])


@pytest.mark.parametrize("name", ["odd", "ranks-zigzag", "ranks-contiguous", "one-token-b5"])
def test_checked_build(cuda_device, monkeypatch, name):
    """The build with device address checks finds nothing to report."""
    monkeypatch.setattr(ops, "LIB_PATH", ops.CHECKED_LIB_PATH)
    monkeypatch.setattr(ops, "_lib", None)
    c = _make(name)
    ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], **_place(c))
    ops.qk_norm_rope_bwd(c["w"], c["opts"], c["q"], c["k"], *[_lay(c, g) for g in c["grads"]], **_place(c))
    assert ops.loong_get_device_status() == ops.LOONG_OK


@pytest.mark.parametrize("name", ["odd-heads-d64", "part-48-inter", "many-heads", "no-norm", "one-token", "two-tokens"])
def test_checked_build_of_heads_that_do_not_fill_a_warp(cuda_device, monkeypatch, name):
    """Every address a lane copies from or stores to lies in its tensor, those of lanes past the last head too."""
    monkeypatch.setattr(ops, "LIB_PATH", ops.CHECKED_LIB_PATH)
    monkeypatch.setattr(ops, "_lib", None)
    c = _make(name)
    got = ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], **_place(c))
    ops.qk_norm_rope_bwd(c["w"], c["opts"], c["q"], c["k"], *[_lay(c, g) for g in c["grads"]], **_place(c))
    assert ops.loong_get_device_status() == ops.LOONG_OK
    assert torch.equal(got[2].view(torch.int16), _lay(c, c["v"]).view(torch.int16))


def test_stream_as_a_number(cuda_device):
    """The calls take a cudaStream_t as a number too, as loong_attn_fwd does: a stream's, 0 and 1 (the legacy
    default stream)."""
    from head_context_attention_gb300.ops import attn_bias_bwd, attn_bias_fwd, log_buckets
    c = _make("ranks-zigzag")
    dy = [_lay(c, g) for g in c["grads"]]
    buckets, t = log_buckets(8, 40), torch.randn((8, 8), device="cuda").to(torch.bfloat16)

    def run(stream):
        q, k, v = ops.qk_norm_rope(c["w"], c["opts"], c["q"], c["k"], c["v"], stream=stream, **_place(c))
        o, lse, res = attn_bias_fwd(c["w"], q, k, v, t, buckets, layout=c["layout"], stream=stream)
        _, dk, dv, dt = attn_bias_bwd(c["w"], q, k, v, o, lse, o, t, buckets, o_res=res, layout=c["layout"],
                                      stream=stream)
        return (q, k, v, o, lse, dk, dv, dt) + ops.qk_norm_rope_bwd(c["w"], c["opts"], c["q"], c["k"], *dy,
                                                                    stream=stream, **_place(c))
    want = run(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for number in (side.cuda_stream, 0, 1):
        got = run(number)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), number


def test_angles_of_any_position(cuda_device):
    """Angles of positions up to 2^55, of frequencies of both signs, against decimals of 60 digits: the stated
    2^-23 + |position| (|inv_freq| 2^-52 + 2 pi 2^-64) of a radian; then sincospi's and the product's 2^-22 and a
    rounding to bf16."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    freqs = [1.0, -1.0, 1e-2, -1e-2, 500000.0 ** -0.98, -(500000.0 ** -0.98), 3.7e-7, -3.7e-7]
    pos = [2 ** 45 + 12345, -(2 ** 45) - 777, 2 ** 50 + 3, 2 ** 55 - 1, 5 * 2 ** 52 + 99, -(2 ** 53), 2 ** 31 - 1, 131072]
    w = inputs.small(len(pos), 1, 1, 64, placement=0)
    q = torch.zeros((1, len(pos), 1, 64), device="cuda", dtype=torch.bfloat16)
    q[..., :8] = 1    # pairs (i, i + 8): (1, 0) turns to (cos, sin)
    opts = ops.make_qk_opts(64, norm=False, rot_dim=16, inv_freq=freqs)
    y, _, _ = ops.qk_norm_rope(w, opts, q, q, positions=torch.tensor([pos], device="cuda"))
    y = to64(y[0, :, 0])
    for t, p in enumerate(pos):
        for i, f in enumerate(freqs):
            angle = float(Decimal(p) * Decimal(f) % two_pi)
            tol = 2.0 ** -23 + abs(p) * (abs(f) * 2.0 ** -52 + 2 * np.pi * 2.0 ** -64) + 2.0 ** -22
            for got, want in ((y[t, i], np.cos(angle)), (y[t, i + 8], np.sin(angle))):
                assert abs(got - want) <= tol + 2.0 ** -8 * (abs(want) + tol), (p, f, got, want, tol)
