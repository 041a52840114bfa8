"""The masked and the paged attention in less usual surroundings: the library with
address checks, long sequences and far offsets, timing events, several host
threads, and one layer trained and then answering."""
import threading

import numpy as np
import pytest
import torch

from head_context_attention_gb300 import inputs, ops
from oracle import mask as omask
from tests.helpers import to64
from tests.test_gpu_checked import _library
from tests.test_gpu_layout import _within_one_bf16_spacing
from tests.test_gpu_mask_attn import _check, _make, _pack, _run
from tests.test_gpu_paged_attn import _Setup

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("layout", [ops.LAYOUT_NATURAL, ops.LAYOUT_RANK_MAJOR])
@pytest.mark.parametrize("name", ["one-token-padded", "ragged-blocks", "prefix", "random-causal-ring", "nothing",
                                  "one-head-tile-pairs", "group-of-34", "cap-saturated", "flushes"])
def test_checked_library_trips_no_check(cuda_device, name, layout):
    w, x, r, cap = _make(name)
    if layout == ops.LAYOUT_RANK_MAJOR:
        x = _pack(w, x)
    want = _run(w, x, r, cap, layout=layout)
    with _library(ops.CHECKED_LIB_PATH):
        got = _run(w, x, r, cap, layout=layout)   # asks for the device's status
    for i in (0, 1, 3, 4):   # O, LSE, dK, dV
        assert torch.equal(_bits(got[i]), _bits(want[i])), i
    assert _within_one_bf16_spacing(got[2], want[2])


@pytest.mark.parametrize("name", ["one-key", "token-tile-ends", "group-of-three", "chunk", "window", "many"])
def test_checked_library_paged(cuda_device, name):
    s = _Setup(name)
    want = s.run()
    with _library(ops.CHECKED_LIB_PATH):
        got = s.run()
        s.check(*got)
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want))


def test_long_sequence_of_documents(cuda_device):
    """131,072 tokens of packed documents: some of them against the oracle, which needs only the document."""
    S, hq, hkv, d, cap = 131072, 4, 2, 64, 25.0
    w = inputs.Workload("long", S, hq, hkv, d, 2, 8, 4, 2, True)
    x = inputs.make_inputs(w, device="cuda")
    rng = np.random.default_rng(5)
    lengths = []
    while sum(lengths) < S - 1000:
        lengths.append(int(rng.integers(1, 9000)))
    lengths = lengths[:-1]
    r = ops.document_ranges([lengths], S)
    out = _run(w, x, r, cap)
    starts = np.concatenate([[0], np.cumsum(lengths)])
    short = [i for i, n in enumerate(lengths) if n < 1500]
    for i in (short[0], short[-1], len(lengths) - 1):
        a, b = int(starts[i]), int(min(starts[i] + 1500, starts[i + 1]))
        whole = b == starts[i + 1]
        n = b - a
        t = omask.forward_backward(*(to64(x[m][0, a:b]) for m in ("q", "k", "v", "do")),
                                   omask.sees(np.tile([0, n], (n, 1)), n, True), ops.default_scale(d), cap)
        assert np.abs(to64(out[0][0, a:b]) - t["o"]).max() <= 2e-2
        assert np.abs(to64(out[1][0, :, a:b]) - t["lse"]).max() <= 1e-3
        assert np.all(np.abs(to64(out[2][0, a:b]) - t["dq"]) <= 5e-2 * (1 + np.abs(t["dq"])))
        if whole:   # the keys' gradients need the whole document
            for got, m in ((out[3], "dk"), (out[4], "dv")):
                assert np.all(np.abs(to64(got[0, a:b]) - t[m]) <= 5e-2 * (1 + np.abs(t[m]))), m
    pad = int(starts[-1])
    assert bool((out[0][0, pad:] == 0).all()) and bool(torch.isneginf(out[1][0, :, pad:]).all())
    assert all(bool((g[0, pad:] == 0).all()) for g in out[2:])


@pytest.mark.parametrize("B,S,hq,hkv,d,cp,causal,cap", [
    (14, 900, 6, 2, 64, 1, True, 0.0), (14, 900, 6, 2, 128, 1, True, 15.0), (20, 500, 8, 4, 128, 2, False, 0.0),
    (9, 700, 16, 2, 64, 1, False, 30.0), (40, 130, 5, 5, 128, 1, True, 0.0)])
def test_more_tiles_than_multiprocessors(cuda_device, B, S, hq, hkv, d, cp, causal, cap):
    """Several query tiles a block one after the other, some of which see nothing in between."""
    w = inputs.Workload("many", S, hq, hkv, d, 1, cp, cp, 1, True, placement=0, batch=B, causal=causal)
    x = inputs.make_inputs(w, device="cuda")
    rng = np.random.default_rng(S)
    docs = [[] if b % 3 == 1 else [int(n) for n in rng.integers(1, S // 3, 2 + b % 2)] for b in range(B)]
    r = ops.document_ranges(docs, S, causal=causal)
    out = _run(w, x, r, cap)
    _check(w, x, r, cap, out)
    # another order of the blocks, and padding that is not finite, change no bit
    pad = torch.zeros((B, S), dtype=torch.bool)
    for b, lengths in enumerate(docs):
        pad[b, sum(lengths):] = True
    x = {n: t.masked_fill(pad.cuda()[..., None, None], float("nan")) for n, t in x.items()}
    for _ in range(3):
        again = _run(w, x, r, cap)
        for i in (0, 1, 3, 4):
            assert torch.equal(_bits(again[i]), _bits(out[i])), i


@pytest.mark.parametrize("B,S,hq,hkv,d,cap", [(4, 900, 6, 2, 64, 20.0), (2, 1500, 9, 3, 128, 5.0), (5, 777, 8, 8, 64, 0.0)])
def test_two_uneven_tiles_a_multiprocessor(cuda_device, B, S, hq, hkv, d, cap):
    w = inputs.Workload("uneven", S, hq, hkv, d, 1, 1, 1, 1, True, placement=0, batch=B)
    x = inputs.make_inputs(w, device="cuda")
    out = _run(w, x, None, cap)
    _check(w, x, None, cap, out)
    again = _run(w, x, None, cap)
    for i in (0, 1, 3, 4):
        assert torch.equal(_bits(again[i]), _bits(out[i])), i


def test_pool_past_32_bits(cuda_device):
    """A pool of more than 2^32 bytes and 2^31 elements, the sequences' pages at its end."""
    hkv, d, page = 8, 128, 256
    pages = (1 << 31) // (page * hkv * d) + 40
    pool = [torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    n, new = 3000, 5
    used = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(1)
    table = (pages - 1 - torch.randperm(used, generator=g, device="cuda")).to(torch.int32)[None]
    q = torch.randn((new, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((n, hkv, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    for x, p in ((k, pool[0]), (v, pool[1])):
        rows = torch.full((used * page, hkv, d), float("nan"), device="cuda").to(torch.bfloat16)
        rows[:n - new] = x[:n - new]
        p[table[0].long()] = rows.view(used, page, hkv, d)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    o, lse = ops.paged_attn(q, *pool, table, torch.tensor([n], **i32), torch.tensor([0, new], **i32), k=k[-new:],
                            v=v[-new:])
    assert ops.loong_get_device_status() == ops.LOONG_OK
    i = np.arange(n - new, n)
    t = omask.forward_backward(to64(q), to64(k), to64(v), None, omask.sees(np.stack([0 * i, i + 1], 1), n, False),
                               ops.default_scale(d), terms=True)
    assert np.all(np.abs(to64(o) - t["o"]) <= 2.0 ** -8 * np.abs(t["o"]) + 2.0 ** -6 * t["abs_o"])
    assert np.abs(to64(lse) - t["lse"]).max() <= 1e-4
    for x, p in ((k, pool[0]), (v, pool[1])):
        assert torch.equal(p[table[0].long()].view(-1, hkv, d)[:n], x)


def test_timing_events(cuda_device):
    """Events around the main kernels, between a preparation and the launch that follows it."""
    w, x, r, cap = _make("gqa")
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    b.record()
    want = _run(w, x, r, cap)
    ops.loong_set_timing_events(a, b)
    try:
        got = _run(w, x, r, cap)
    finally:
        ops.loong_set_timing_events()
    torch.cuda.synchronize()
    assert 0 < a.elapsed_time(b) < 1000
    for i in (0, 1, 3, 4):
        assert torch.equal(_bits(got[i]), _bits(want[i])), i


def test_several_host_threads(cuda_device):
    """Calls from several threads, each on a stream of its own."""
    w, x, r, cap = _make("gqa")
    s = _Setup("tokens-ragged")
    want, want_paged = _run(w, x, r, cap), s.run()
    rc = r.cuda()
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    if n % 2:
                        o, lse, res = ops.attn_mask_fwd(w, x["q"], x["k"], x["v"], rc, cap)
                        _, dk, dv = ops.attn_mask_bwd(w, x["q"], x["k"], x["v"], o, lse, x["do"], rc, cap, o_res=res)
                        same = [torch.equal(_bits(p), _bits(q)) for p, q in zip((o, lse, dk, dv),
                                                                               (*want[:2], *want[3:]))]
                    else:
                        same = [torch.equal(_bits(p), _bits(q)) for p, q in zip(s.run(append=False), want_paged)]
                    if not all(same):
                        wrong.append((n, same))
        except Exception as e:  # noqa: BLE001
            wrong.append((n, e))
    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[:3]


def test_gradient_of_a_layer_that_then_answers(cuda_device):
    """Two documents and padding through norm + rotation, masked and capped attention and back; then each document's
    last tokens through the cache: the same outputs."""
    hq, hkv, d, S, cap = 4, 2, 128, 260, 30.0
    lengths = [150, 90]
    w = inputs.Workload("layer", S, hq, hkv, d, 1, 1, 1, 1, True, placement=0)
    n = (hq * d, hkv * d, hkv * d)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((1, S, sum(n)), generator=g, device="cuda").to(torch.bfloat16)
    split = lambda y: [t.unflatten(2, (-1, d)) for t in y.split(n, dim=2)]  # noqa: E731
    pos = torch.cat([torch.arange(k) for k in (*lengths, S - sum(lengths))])[None].cuda()
    opts, r = ops.make_qk_opts(d), ops.document_ranges([lengths], S, device="cuda")
    q, k, v = ops.qk_norm_rope(w, opts, *split(x), positions=pos)
    o, lse, res = ops.attn_mask_fwd(w, q, k, v, r, cap)
    do = torch.randn((1, S, hq, d), generator=g, device="cuda").to(torch.bfloat16)
    dx = torch.empty_like(x)
    ops.qk_norm_rope_bwd(w, opts, *split(x)[:2], *ops.attn_mask_bwd(w, q, k, v, o, lse, do, r, cap, o_res=res),
                         positions=pos, into=split(dx))
    assert bool(torch.isfinite(dx.float()).all()) and bool((dx[0, sum(lengths):] == 0).all())
    assert bool((dx[0, :sum(lengths)] != 0).any(-1).all())
    # the directional derivative of the whole layer, by central differences of the calls themselves
    step = torch.randn((1, S, sum(n)), generator=g, device="cuda")
    f = []
    for sign in (1, -1):
        y = (x.float() + sign * 0.0625 * step).to(torch.bfloat16)
        qkv = ops.qk_norm_rope(w, opts, *split(y), positions=pos)
        oo, _, rr = ops.attn_mask_fwd(w, *qkv, r, cap)
        f.append((((oo.double() + rr.double()) * do.double()).sum(), y.double()))
    want = (f[0][0] - f[1][0]).item()
    got = (dx.double() * (f[0][1] - f[1][1])).sum().item()
    # A derivative along random steps is |dx| times their size, give or take; of that the third order of steps of 1/16
    # is about 1 % (1/256 / 6 of derivatives some times the first), the rounding of dx 2^-8, O's error of 2^-12 a term
    # over 123,000 terms of random signs less than 1 %.
    size = dx.double().norm().item() * (f[0][1] - f[1][1]).square().mean().sqrt().item()
    assert abs(got - want) <= 0.05 * size
    i32 = {"dtype": torch.int32, "device": "cuda"}
    kp = torch.full((40, 8, hkv, d), float("nan"), device="cuda").to(torch.bfloat16)
    vp = kp.clone()
    table = torch.arange(40, **i32).view(2, 20)
    qs, ks, vs = (torch.cat([t[0, a:b] for a, b in ((0, 150), (150, 240))]) for t in (q, k, v))
    o2, lse2 = ops.paged_attn(qs, kp, vp, table, torch.tensor(lengths, **i32), torch.tensor([0, 150, 240], **i32), k=ks,
                              v=vs, score_cap=cap)
    assert ops.loong_get_device_status() == ops.LOONG_OK
    assert (o2.float() - o[0, :240].float()).abs().max() <= 2.0 ** -5
    assert (lse2 - lse[0, :, :240]).abs().max() <= 2.0 ** -12

