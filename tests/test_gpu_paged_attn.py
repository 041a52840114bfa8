"""Attention of new tokens over a paged cache against the float64 oracle.

Tolerances, per element (half steps: bf16 2^-8 of the value, fp32 2^-24): a
logit's error dx and the factor 1 + e of every P as in test_gpu_mask_attn.  P is
rounded to bf16 (2^-8), and O divided by the sum of the rounded values: O is off by
at most 2 (2^-8 + e) of A = P |V| (numerator and denominator), sums in fp32 2^-16,
O's own rounding 2^-8 |O|; the LSE's sum is of the values before rounding: e + 2^-22
(1 + |LSE|).
"""
import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import mask as omask
from tests.helpers import to64
from tests.test_gpu_mask_attn import _within

pytestmark = pytest.mark.gpu

# hq, hkv, d, page, window, cap, factor of q, sequences (length with the new tokens, new tokens)
CASES = {
    "one-key": (2, 1, 64, 16, 0, 0, 1, [(1, 1)]),
    "one-key-each": (4, 4, 128, 8, 0, 5, 1, [(1, 1)] * 5),
    "token": (32, 8, 128, 64, 0, 0, 1, [(300, 1)]),
    "token-tile-ends": (4, 2, 64, 128, 0, 0, 1, [(127, 1), (128, 1), (129, 1), (256, 1), (257, 1)]),
    "tokens-ragged": (8, 2, 128, 16, 0, 30, 3, [(700, 1), (3, 1), (129, 1), (1, 1), (1000, 1), (64, 1), (65, 1)]),
    "long-token": (8, 2, 64, 32, 0, 0, 1, [(20000, 1)]),
    "one-head-groups": (6, 6, 128, 32, 0, 0, 1, [(500, 1), (90, 3)]),
    "group-of-34": (34, 1, 64, 16, 0, 0, 1, [(300, 5), (70, 70)]),
    "group-of-three": (12, 4, 64, 16, 0, 15, 3, [(500, 40), (44, 44), (200, 1)]),
    "group-of-128": (128, 1, 128, 16, 0, 0, 1, [(200, 3)]),
    "whole-prompts": (4, 2, 64, 64, 0, 0, 1, [(100, 100), (1, 1), (300, 300)]),
    "chunk": (8, 2, 128, 128, 0, 50, 3, [(1500, 700)]),
    "chunk-d64": (8, 2, 64, 16, 0, 0, 1, [(1500, 700)]),
    "chunk-one-head": (3, 3, 128, 256, 0, 0, 1, [(1100, 600)]),
    "nothing-new": (4, 2, 64, 16, 0, 0, 1, [(50, 0), (70, 2), (0, 0), (9, 1), (33, 0)]),
    "window": (8, 2, 128, 16, 100, 0, 1, [(1000, 1), (90, 90), (500, 300), (101, 1), (100, 1)]),
    "window-one": (4, 2, 64, 8, 1, 0, 1, [(300, 1), (200, 200)]),
    "window-d64-chunk": (16, 2, 64, 32, 300, 20, 3, [(2000, 900)]),
    "page-1024": (4, 2, 128, 1024, 0, 0, 1, [(1500, 1), (1024, 2), (2049, 3)]),
    "many": (4, 1, 64, 16, 0, 0, 1, [(1 + 37 * i % 401, 1) for i in range(300)]),
    "mixed-many": (8, 2, 128, 64, 0, 0, 1, [(1 + 37 * i % 401, min(1 + 37 * i % 401, 1 + 11 * i % 60)) for i in range(70)]),
    "cap-saturated": (4, 2, 64, 16, 0, 2, 40, [(300, 1), (150, 150)]),
    "peaked": (4, 2, 128, 16, 0, 0, 20, [(700, 1), (600, 300)]),
}


class _Setup:
    def __init__(self, name, seed=0, fill=float("nan"), spare=5):
        self.hq, self.hkv, self.d, self.page, self.window, cap, mul, self.seqs = CASES[name]
        self.cap = float(cap)
        g = torch.Generator(device="cuda").manual_seed(100 + seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        used = [-(-n // self.page) for n, _ in self.seqs]
        total = sum(used) + spare
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(used), max(used) + 1), -7, dtype=torch.int32, device="cuda")
        # the pool holds `fill` wherever no sequence keeps a token
        self.kp = torch.full((total, self.page, self.hkv, self.d), fill, dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        self.ks, self.vs, at = [], [], 0
        for b, ((n, new), p) in enumerate(zip(self.seqs, used)):
            self.table[b, :p] = order[at:at + p]
            k, v = rnd(n, self.hkv, self.d), rnd(n, self.hkv, self.d)
            for x, pool in ((k, self.kp), (v, self.vp)):
                rows = pool[order[at:at + p].long()].reshape(-1, self.hkv, self.d)
                rows[:n - new] = x[:n - new]
                pool[order[at:at + p].long()] = rows.view(p, self.page, self.hkv, self.d)
            self.ks.append(k)
            self.vs.append(v)
            at += p
        new = [n for _, n in self.seqs]
        self.tokens = sum(new)
        self.q = (rnd(self.tokens, self.hq, self.d).float() * mul).to(torch.bfloat16)
        self.k = torch.cat([k[len(k) - n:] for k, n in zip(self.ks, new)])
        self.v = torch.cat([v[len(v) - n:] for v, n in zip(self.vs, new)])
        self.lens = torch.tensor([n for n, _ in self.seqs], dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")

    def run(self, append=True, **kw):
        k, v = (self.k, self.v) if append else (None, None)
        return ops.paged_attn(self.q, self.kp, self.vp, self.table, self.lens, self.starts, k=k, v=v,
                              window=self.window, score_cap=self.cap, **kw)

    def check(self, o, lse):
        assert ops.loong_get_device_status() == ops.LOONG_OK
        at = 0
        for b, (n, new) in enumerate(self.seqs):
            i = np.arange(n - new, n)
            first = np.maximum(i - self.window + 1, 0) if self.window else 0 * i
            see = omask.sees(np.stack([first, i + 1], 1), n, False)
            t = omask.forward_backward(to64(self.q[at:at + new]), to64(self.ks[b]), to64(self.vs[b]), None, see,
                                       ops.default_scale(self.d), self.cap, terms=True)
            L = t["logit"].max(initial=0)
            dx = (self.d + 4) * 2.0 ** -24 * L + 2.0 ** -21 * self.cap
            e = 2 * (dx + 2.0 ** -21 + 2.0 ** -23 * (min(L, self.cap) if self.cap else L))
            _within(f"O of sequence {b}", o[at:at + new], t["o"],
                    2.0 ** -8 * np.abs(t["o"]) + (2 * (2.0 ** -8 + e) + 2.0 ** -16) * t["abs_o"])
            _within(f"LSE of sequence {b}", lse[:, at:at + new], t["lse"],
                    e + 2.0 ** -22 * (1 + np.abs(t["lse"])))
            at += new


@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(cuda_device, name):
    s = _Setup(name)
    before = s.kp.clone(), s.vp.clone()
    o, lse = s.run()
    s.check(o, lse)
    # the pages hold the new tokens, and nothing else of them changed
    for pool, old, seqs in ((s.kp, before[0], s.ks), (s.vp, before[1], s.vs)):
        for b, (n, new) in enumerate(s.seqs):
            pages = s.table[b, :-(-n // s.page)].long()
            assert torch.equal(pool[pages].reshape(-1, s.hkv, s.d)[:n].view(torch.int16), seqs[b].view(torch.int16))
            rows = old[pages].reshape(-1, s.hkv, s.d)
            rows[n - new:n] = seqs[b][n - new:]
            old[pages] = rows.view(-1, s.page, s.hkv, s.d)
        assert torch.equal(pool.view(torch.int16), old.view(torch.int16))
    # the same bits again, the tokens being there already
    o2, lse2 = s.run(append=False)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))


def test_after_the_projection(cuda_device):
    """A layer's steps in order: projection -> norm and rotation -> cache and attention, in two chunks and then a token
    at a time; the outputs are the masked attention's over the whole sequence at once, both to their roundings."""
    hq, hkv, d, S, page, cap, window = 8, 2, 64, 333, 16, 20.0, 150
    n = (hq * d, hkv * d, hkv * d)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, S, sum(n)), generator=g, device="cuda").to(torch.bfloat16)
    split = lambda y: [t.unflatten(2, (-1, d)) for t in y.split(n, dim=2)]  # noqa: E731
    opts = ops.make_qk_opts(d)

    def project(at, to):
        w = inputs.Workload("step", to - at, hq, hkv, d, 1, 1, 1, 1, False, placement=0)
        q, k, _ = ops.qk_norm_rope(w, opts, *split(x[:, at:to])[:2], pos_begin=at)
        return q[0], k[0], split(x[:, at:to])[2][0]  # V as it lies in the projection
    w = inputs.Workload("whole", S, hq, hkv, d, 1, 1, 1, 1, False, placement=0)
    q, k, v = project(0, S)
    r = ops.document_ranges([[S]], S, window=window, device="cuda")
    want, want_lse, _ = ops.attn_mask_fwd(w, q[None], k[None], v[None].contiguous(), r, cap)
    pages = -(-S // page)
    kp = torch.full((pages + 2, page, hkv, d), float("nan"), device="cuda").to(torch.bfloat16)
    vp = kp.clone()
    table = torch.randperm(pages + 2, generator=g, device="cuda").to(torch.int32)[None, :pages].contiguous()
    at = 0
    for to in [200, 290] + list(range(291, S + 1)):
        q, k, v = project(at, to)
        o, lse = ops.paged_attn(q, kp, vp, table, torch.tensor([to], dtype=torch.int32, device="cuda"),
                                torch.tensor([0, to - at], dtype=torch.int32, device="cuda"), k=k, v=v, window=window,
                                score_cap=cap)
        assert (o.float() - want[0, at:to].float()).abs().max() <= 2.0 ** -5  # |V| up to 4.5: 3 * 2^-8 of it
        assert (lse - want_lse[0, :, at:to]).abs().max() <= 2.0 ** -7
        at = to
    assert ops.loong_get_device_status() == ops.LOONG_OK


@pytest.mark.parametrize("name", ["tokens-ragged", "group-of-three", "window", "chunk"])
def test_graph_replays_on_other_lengths(cuda_device, name):
    """A captured call, replayed as the sequences grow."""
    s = _Setup(name)
    o, lse = s.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = s.run()
    graph.replay()
    torch.cuda.synchronize()
    s.check(o, lse)
    # other new tokens, the last of shorter sequences
    rng = np.random.default_rng(1)
    seqs, at = [], 0
    for b, (n, new) in enumerate(s.seqs):
        cut = int(rng.integers(0, n - new + 1))
        seqs.append((n - cut, new))
        s.ks[b], s.vs[b] = s.ks[b][:n - cut], s.vs[b][:n - cut]
        s.k[at:at + new], s.v[at:at + new] = s.ks[b][n - cut - new:], s.vs[b][n - cut - new:]
        at += new
    s.seqs = seqs
    s.lens.copy_(torch.tensor([n for n, _ in seqs], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    s.check(o, lse)


def test_two_graphs_and_streams(cuda_device):
    a, b = _Setup("tokens-ragged"), _Setup("group-of-three")
    outs = []
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(s.run())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for s, out in zip((a, b), outs):
        s.check(*out)
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        out = a.run(stream=stream)
        st.synchronize()
        a.check(*out)


def test_strided_inputs(cuda_device):
    s = _Setup("group-of-three")
    fused = torch.cat([x.flatten(1) for x in (s.q, s.k, s.v)], 1)
    n = (s.hq * s.d, s.hkv * s.d, s.hkv * s.d)
    s.q, s.k, s.v = (x.unflatten(1, (-1, s.d)) for x in fused.split(n, 1))
    s.check(*s.run())


def test_rows_behind_the_last_sequence(cuda_device):
    """A padded batch: rows behind the last sequence, and before the first, stay as they were."""
    s = _Setup("group-of-three")
    pad = lambda x, v: torch.cat([torch.full_like(x[:3], v), x, torch.full_like(x[:9], v)])  # noqa: E731
    nan = float("nan")
    k, v = pad(s.k, nan), pad(s.v, nan)
    q = pad(s.q, nan)
    out = torch.full((len(q), s.hq, s.d), 7.0, device="cuda").to(torch.bfloat16), torch.full((s.hq, len(q)), 7.0, device="cuda")
    before = s.kp.clone()
    o, lse = ops.paged_attn(q, s.kp, s.vp, s.table, s.lens, s.starts + 3, k=k, v=v, window=s.window, score_cap=s.cap,
                            out=out)
    assert o is out[0] and lse is out[1]
    s.check(o[3:3 + s.tokens], lse[:, 3:3 + s.tokens])
    for rows in (slice(0, 3), slice(3 + s.tokens, None)):
        assert bool((o[rows] == 7).all()) and bool((lse[:, rows] == 7).all())
    spare = torch.ones(len(s.kp), dtype=torch.bool, device="cuda")
    for b, (n, _) in enumerate(s.seqs):
        spare[s.table[b, :-(-n // s.page)].long()] = False
    assert torch.equal(s.kp[spare].view(torch.int16), before[spare].view(torch.int16))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["chunk", "window", "group-of-34"])
def test_values_that_are_not_finite(cuda_device, name, value):
    """One in V reaches the tokens that see its key, as NaN, and no others; one in K likewise."""
    for kind in ("v", "k"):
        s = _Setup(name, fill=0.0)
        b = len(s.seqs) - 1 if name == "window" else int(np.argmax([n for _, n in s.seqs]))
        n, new = s.seqs[b]
        at = n - max(new // 2, 1)
        (s.v if kind == "v" else s.k)[sum(m for _, m in s.seqs[:b]) + at - (n - new), 0, 5] = value
        clean = _Setup(name, fill=0.0).run()
        o, lse = s.run()
        assert ops.loong_get_device_status() == ops.LOONG_OK
        i = torch.arange(n - new, n, device="cuda")
        sees = (i >= at) & ((i < at + s.window) if s.window else torch.ones_like(i, dtype=torch.bool))
        hit = torch.zeros(s.tokens, dtype=torch.bool, device="cuda")
        t0 = sum(m for _, m in s.seqs[:b])
        hit[t0:t0 + new] = sees
        g = s.hq // s.hkv
        # An infinite K's score is beyond the cap's polynomial, so the rows of its warp take the other form of tanh:
        # both are within their bound of the exact value (see the top; A <= |V|max, e < 2^-12 here), so within twice
        # 2^-8 |O| + 2 (2^-8 + 2^-12) |V|max of each other.  Everything else is the same bits.
        capped = s.cap and kind == "k"
        far = 2.0 ** -7 * clean[0].float().abs() + 4 * (2.0 ** -8 + 2.0 ** -12) * s.v[torch.isfinite(s.v)].abs().max()
        same = (o.float() - clean[0].float()).abs() <= far if capped else o == clean[0]
        assert bool(same[~hit].all()) and bool(same[:, g:].all())
        if kind == "v" or not (s.cap and value == float("inf")):
            bad = ~torch.isfinite(o[hit][:, :g].float()).all(-1)
            assert bool(bad.all()) if kind == "v" or value != value else bool(bad.any())


def test_wrong_pages_and_lengths_are_reported(cuda_device):
    """A page outside the pool, lengths beyond the table, starts out of order: reported, nothing outside the tensors
    is touched, and the next call is as ever."""
    for what in ("page", "negative page", "length", "negative length", "short", "starts", "starts beyond"):
        s = _Setup("tokens-ragged", fill=0.0)
        if what == "page":
            s.table[0, 1] = 10 ** 6
        elif what == "negative page":
            s.table[0, 0] = -1
        elif what == "length":
            s.lens[0] = 10 ** 7
        elif what == "negative length":
            s.lens[2] = -5
        elif what == "short":
            s.lens[3] = 0
        elif what == "starts":
            s.starts[2] = 0
        else:
            s.starts[-1] = 10 ** 6
        s.run()
        assert ops.loong_get_device_status() == ops.LOONG_ERR_DEVICE_CHECK, what
        t = _Setup("tokens-ragged")
        t.check(*t.run())


def test_refusals(cuda_device):
    s = _Setup("group-of-three")
    call = lambda **kw: ops.paged_attn(**({"q": s.q, "k_pages": s.kp, "v_pages": s.vp, "table": s.table,  # noqa: E731
                                           "lens": s.lens, "starts": s.starts, "k": s.k, "v": s.v} | kw))
    for kw, what in (({"q": s.q.float()}, "q must be"), ({"lens": s.lens.long()}, "lens"),
                     ({"starts": s.starts[:-1]}, "starts"), ({"table": s.table.cpu()}, "table"),
                     ({"k": None}, "belong together"), ({"v": s.v[:-1]}, "v must be"),
                     ({"q": s.q[:1].expand(s.tokens, -1, -1)}, "overlap"),
                     ({"k": s.k.transpose(1, 2).contiguous().transpose(1, 2)}, "contiguous heads"),
                     ({"v_pages": s.vp[:-1]}, "v_pages"), ({"table": s.table[0]}, "table")):
        with pytest.raises(ValueError, match=what):
            call(**kw)
    for kw in ({"window": -1}, {"score_cap": -1.0}, {"score_cap": float("nan")}):
        with pytest.raises(ops.LoongError):
            call(**kw)
    empty = call(q=s.q[:0], k=s.k[:0], v=s.v[:0])
    assert empty[0].shape == (0, s.hq, s.d) and empty[1].shape == (s.hq, 0)
