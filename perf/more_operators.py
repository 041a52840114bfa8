"""Workloads of the masked, the capped and the paged attention.

Three operators:

* ``mask`` forward and training step: ring attention in which every query sees
  a range of keys of its own (packed documents, prefixes that see themselves
  whole, windows, padding that sees nothing) and whose scaled scores may be
  capped, cap * tanh(score / cap).
* ``paged``: new tokens of several sequences (one each, a chunk, or a mixture)
  are written into a cache of pages and attend over what their sequence has
  there, with the same cap and an optional window.

A case is a dict of plain values.  ``prepare`` makes its inputs, ``run`` makes
one pass, in elementary torch operations or (``own``) through the package.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def _mask(name, kind, batch, seqlen, hq, hkv, d, hp=1, cp=1, zigzag=True, rank_major=False, see="causal", doc=0,
          window=0, pad=False, cap=0.0, stepwise=False, cut=1):
    """see: what a token sees of its own document: "causal" (itself and what is
    before it), "prefix" (that, and the document's first part whole) or "whole".
    doc: about how long a document is (0: one per sequence).  pad: the end of
    every sequence belongs to no document.  cut: numbers the documents' lengths."""
    return {"name": name, "op": "mask", "kind": kind, "batch": batch, "seqlen": seqlen, "hq": hq, "hkv": hkv, "d": d,
            "hp": hp, "cp": cp, "zigzag": zigzag, "rank_major": rank_major, "see": see, "doc": doc, "window": window,
            "pad": pad, "cap": cap, "stepwise": stepwise, "cut": cut}


def _paged(name, batch, new, length, hq, hkv, d, page=64, window=0, cap=0.0, even=False, cut=1):
    """length: the longest sequence, its new tokens included; new: the most new
    tokens of one.  even: every sequence has as many of both."""
    return {"name": name, "op": "paged", "batch": batch, "new": new, "length": length, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "window": window, "cap": cap, "even": even, "cut": cut}


def listed():
    return [
        # three short prompts of different lengths, padded to one
        _mask("mask-short", "fwd", 3, 100, 4, 2, 64, zigzag=False, pad=True, cap=30.0),
        # prompts whose first part sees itself whole, heads of their own, capped scores
        _mask("mask-prefix-s4k", "fwd", 2, 4096, 16, 16, 128, zigzag=False, see="prefix", cap=50.0),
        # the 8B layer over packed documents at 32K tokens, on the ranks' layout
        _mask("mask-8b-s32k", "fwd", 1, 32768, 32, 8, 128, hp=4, cp=8, rank_major=True, doc=4096),
        # a training step of the tiny layer over a few documents
        _mask("mask-tiny-s1k-train", "train", 1, 1024, 4, 2, 64, hp=2, cp=4, doc=256),
        # a ragged training step of an encoder over padded documents, blocks that are no multiple of a tile
        _mask("mask-odd-train", "train", 2, 1990, 6, 3, 64, cp=5, see="whole", doc=300, pad=True, cap=20.0),
        # a training step of the 8B layer with capped scores, one document
        _mask("mask-8b-s16k-cap-train", "train", 1, 16384, 32, 8, 128, hp=8, cp=16, rank_major=True, cap=50.0),
        # a training step of the 8B layer over packed documents at 64K tokens
        _mask("mask-8b-s64k-train", "train", 1, 65536, 32, 8, 128, hp=8, cp=16, doc=8192),
        # the next token of one sequence
        _paged("paged-token", 1, 1, 1001, 32, 8, 128, even=True),
        # the next token of 61 sequences of all lengths
        _paged("paged-tokens-b61", 61, 1, 16384, 64, 8, 128),
        # the next token of one very long sequence
        _paged("paged-token-s128k", 1, 1, 131072, 32, 8, 128, page=128, even=True),
        # new tokens of a mixture of sequences, one to hundreds each, through a windowed layer with capped scores
        _paged("paged-mixed-window", 13, 300, 5000, 12, 4, 64, page=16, window=1024, cap=30.0),
        # a chunk of a long prompt of the 8B layer
        _paged("paged-8b-chunk", 1, 2048, 32768, 32, 8, 128, page=128, cap=50.0, even=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.randint(1, 8)
    hq = hkv * rng.randint(1, 8)
    cap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    cut = rng.randint(1, 1 << 20)
    batch = rng.randint(1, 3)
    if rng.random() < 0.45:
        window = rng.choice([0, 0, 0, _log_int(rng, 64, 8192)])
        page = rng.choice([16, 32, 64, 128, 256])
        kind = rng.choice(["token", "mixed", "chunk"])
        if kind == "token":
            batch = _log_int(rng, 1, 128)
            most = min(131072, (1 << 20) * 8 * 128 // (batch * hkv * d))
            return _paged("", batch, 1, _log_int(rng, 16, most), hq, hkv, d, page, window, cap, rng.random() < 0.3, cut)
        if kind == "mixed":
            batch = rng.randint(2, 24)
            length = _log_int(rng, 16, 8192)
            return _paged("", batch, _log_int(rng, 2, min(length, 512)), length, hq, hkv, d, page, window, cap, False,
                          cut)
        length = _log_int(rng, 128, 49152)
        most = max(64, min(length, 2048 * 32768 * 32 * 128 // (length * hq * d)))
        return _paged("", 1, _log_int(rng, 64, min(most, 4096, length)), length, hq, hkv, d, page, window, cap, True,
                      cut)
    cp = rng.choice([1, 1, 2, 3, 4, 8])
    hp = rng.choice([p for p in (1, 1, 2, 4) if hkv % p == 0])
    zigzag = rng.random() < 0.7
    unit = (2 * cp if zigzag else cp) * hp  # the sequence length is a multiple of this
    train = rng.random() < 0.6
    see = rng.choice(["causal", "causal", "prefix", "whole"])
    # scores of a listed pass, half of 32768^2 (forward) or of 16384^2 (training) of 32 heads of 128
    most = (16384 if train else 32768) ** 2 * 32 * 128 // 2
    top = min(65536, math.sqrt(most * (2 if see == "causal" else 1) / (batch * hq * d)))
    s = unit * max(1, _log_int(rng, 20, top) // unit)
    doc = rng.choice([0, _log_int(rng, 16, s + 16), _log_int(rng, 16, s + 16)])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, s + 16)]) if see == "causal" else 0
    return _mask("", "train" if train else "fwd", batch, s, hq, hkv, d, hp, cp, zigzag, rng.random() < 0.5, see, doc,
                 window, rng.random() < 0.3, cap, rng.random() < 0.2, cut)


# ----------------------------------------------------------- shared geometry
def _order(c):
    """Natural token of every position of the ranks' layout, [cp * S/cp]."""
    n = 2 * c["cp"] if c["zigzag"] else c["cp"]
    blk = c["seqlen"] // n
    blocks = []
    for r in range(c["cp"]):
        blocks += [r, n - 1 - r] if c["zigzag"] else [r]
    return torch.cat([torch.arange(b * blk, (b + 1) * blk) for b in blocks])


def _to_layout(c, x):
    """[B, S, H, d] -> the case's layout."""
    if not c["rank_major"]:
        return x
    b, s, h, d = x.shape
    y = x[:, _order(c).to(x.device)].view(b * c["cp"], s // c["cp"], c["hp"], h // c["hp"], d)
    return y.transpose(1, 2).contiguous()


def _from_layout(c, y):
    if not c["rank_major"]:
        return y
    n, p, sr, hr, d = y.shape
    x = torch.empty((n // c["cp"], c["seqlen"], p * hr, d), dtype=y.dtype, device=y.device)
    x[:, _order(c).to(y.device)] = y.transpose(1, 2).reshape(x.shape)
    return x


def _documents(c):
    """For every sequence its documents, (start, length, length of the prefix)."""
    rng = random.Random(c["cut"])
    out = []
    for _ in range(c["batch"]):
        end = c["seqlen"]
        if c["pad"]:
            end -= rng.randint(0, c["seqlen"] // 3)
        docs, at = [], 0
        while at < end:
            n = end - at if not c["doc"] else min(end - at, max(1, _log_int(rng, c["doc"] / 3, c["doc"] * 3)))
            docs.append((at, n, rng.randint(1, n)))
            at += n
        out.append(docs)
    return out


def _ranges(c):
    """The keys [begin, end) that every query sees, int32 [B, S, 2] on the host."""
    r = torch.zeros((c["batch"], c["seqlen"], 2), dtype=torch.int32)
    for b, docs in enumerate(_documents(c)):
        for at, n, prefix in docs:
            t = torch.arange(at, at + n, dtype=torch.int32)
            r[b, at:at + n, 0] = at
            if c["see"] == "whole":
                r[b, at:at + n, 1] = at + n
            else:
                r[b, at:at + n, 1] = t + 1 if c["see"] == "causal" else (t + 1).clamp(min=at + prefix)
            if c["window"]:
                r[b, at:at + n, 0] = (t + 1 - c["window"]).clamp(min=at)
    return r


def _sequences(c):
    """For every sequence of the cache its length and how many tokens of it are new."""
    rng = random.Random(c["cut"])
    out = []
    for _ in range(c["batch"]):
        if c["even"]:
            out.append((c["length"], c["new"]))
            continue
        n = _log_int(rng, max(1, c["length"] // 256), c["length"])
        new = 1 if c["new"] == 1 else min(n, _log_int(rng, 1, c["new"]))
        if c["new"] > 1 and rng.random() < 0.1:
            new = 0  # nothing new this time
        out.append((n, new))
    return out


# ------------------------------------------------------------------ prepare
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    st = {"case": c}
    if c["op"] == "mask":
        b, s = c["batch"], c["seqlen"]
        for n, h in (("q", hq), ("k", hkv), ("v", hkv), ("do", hq)):
            if n != "do" or c["kind"] == "train":
                x = _normal(g, b, s, h, d)
                if n == "q" and c["cap"]:
                    x *= 3  # scores that the cap bends
                st[n] = _to_layout(c, x.to(torch.bfloat16))
        st["host_range"] = _ranges(c)
        # causal descriptors have the end of the range already; a document in one piece needs no range then
        st["range"] = None if c["see"] == "causal" and not (c["doc"] or c["pad"] or c["window"]) else \
            st["host_range"].cuda()
        if own:
            from head_context_attention_gb300 import inputs
            st["w"] = inputs.Workload("mask", s, hq, hkv, d, c["hp"], c["cp"], c["cp"], 1, c["kind"] == "train",
                                      batch=b, placement=1 if c["zigzag"] else 0, causal=c["see"] == "causal")
        return st
    seqs = _sequences(c)
    page = c["page"]
    used = [-(-n // page) for n, _ in seqs]
    total = sum(used) + 3  # the pool has free pages as well
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    st["table"] = torch.zeros((c["batch"], max(used)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        st["table"][b, :n] = order[at:at + n]
        at += n
    st["k_pages"] = torch.empty((total, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    st["v_pages"] = torch.empty_like(st["k_pages"])
    for x in (st["k_pages"], st["v_pages"]):
        x.normal_(generator=g)
    tokens = sum(n for _, n in seqs)
    q = _normal(g, tokens, hq, d)
    st["q"] = (q * 3 if c["cap"] else q).to(torch.bfloat16)
    st["k"] = _normal(g, tokens, hkv, d).to(torch.bfloat16)
    st["v"] = _normal(g, tokens, hkv, d).to(torch.bfloat16)
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    st["lens"] = torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda")
    st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    st["seqs"] = seqs
    return st


# ---------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if own:
        return _own_mask(c, state) if c["op"] == "mask" else _own_paged(c, state)
    return _plain_mask(c, state) if c["op"] == "mask" else _plain_paged(c, state)


def _own_mask(c, st):
    from head_context_attention_gb300 import ops
    how = {"key_range": st["range"], "score_cap": c["cap"],
           "mode": ops.MODE_STEPWISE if c["stepwise"] else ops.MODE_FUSED,
           "layout": ops.LAYOUT_RANK_MAJOR if c["rank_major"] else ops.LAYOUT_NATURAL}
    w, q, k, v = (st[n] for n in ("w", "q", "k", "v"))
    train = c["kind"] == "train"
    o, lse, o_res = ops.attn_mask_fwd(w, q, k, v, res=train, **how)
    if not train:
        return o, lse
    return (o, lse) + ops.attn_mask_bwd(w, q, k, v, o, lse, st["do"], o_res=o_res, **how)


def _own_paged(c, st):
    from head_context_attention_gb300 import ops
    o, lse = ops.paged_attn(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["starts"],
                            k=st["k"], v=st["v"], window=c["window"], score_cap=c["cap"])
    return o, lse, st["k_pages"], st["v_pages"]


# -------------------------------------------------------------- plain forms
def _plain_rows(x, see, cap):
    """Softmax of the scores x [h, n, keys] (overwritten), capped, over the keys
    of ``see`` [n, keys]: (weights, LSE, the cap's derivative or None)."""
    slope = None
    if cap:
        t = torch.tanh(x.div_(cap))
        slope = 1 - t * t
        x = t.mul_(cap)
    x = x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, top + l.log(), -math.inf)
    p = p.div_(torch.where(l > 0, l, 1.0))
    return p, lse.squeeze(-1), slope


def _plain_mask(c, st):
    train, cap = c["kind"] == "train", c["cap"]
    b_, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d)
    names = ("q", "k", "v", "do") if train else ("q", "k", "v")
    nat = {n: _from_layout(c, st[n]) for n in names}
    o = torch.zeros((b_, s, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b_, hq, s), -math.inf, device="cuda")
    if train:
        dq = torch.zeros_like(o)
        dk, dv = torch.empty_like(nat["k"]), torch.empty_like(nat["v"])
    rows = max(1, min(s, (1 << 27) // (hq * s)))
    host = st["host_range"]
    t = torch.arange(s, device="cuda")
    for b in range(b_):
        k = nat["k"][b].transpose(0, 1).float()  # [hkv, S, d]
        v = nat["v"][b].transpose(0, 1).float()
        if st["range"] is None:
            first, last = torch.zeros_like(t), t + 1
        else:
            first, last = st["range"][b, :, 0], st["range"][b, :, 1]
        if train:
            dk32, dv32 = torch.zeros_like(k), torch.zeros_like(v)
        for i0 in range(0, s, rows):
            i1 = min(s, i0 + rows)
            n = i1 - i0
            r = host[b, i0:i1]
            r = r[r[:, 0] < r[:, 1]]
            if not len(r):
                continue
            k0, k1 = int(r[:, 0].min()), int(r[:, 1].max())
            q = nat["q"][b, i0:i1].float().transpose(0, 1).reshape(hkv, g * n, d)
            kc, vc = k[:, k0:k1], v[:, k0:k1]
            x = (q @ kc.transpose(1, 2)).mul_(scale).view(hq, n, k1 - k0)
            j = t[k0:k1]
            see = (j >= first[i0:i1, None]) & (j < last[i0:i1, None])
            p, lse[b, :, i0:i1], slope = _plain_rows(x, see, cap)
            p = p.view(hkv, g * n, k1 - k0)
            o32 = p @ vc
            o[b, i0:i1] = o32.view(hq, n, d).transpose(0, 1)
            if not train:
                continue
            do = nat["do"][b, i0:i1].float().transpose(0, 1).reshape(hkv, g * n, d)
            dv32[:, k0:k1] += p.transpose(1, 2) @ do
            ds = do @ vc.transpose(1, 2)
            ds = ds.sub_((do * o32).sum(-1, keepdim=True)).mul_(p)
            if cap:
                ds.mul_(slope.view(ds.shape))
            dq[b, i0:i1] = (ds @ kc).mul_(scale).view(hq, n, d).transpose(0, 1)
            dk32[:, k0:k1] += (ds.transpose(1, 2) @ q).mul_(scale)
        if train:
            dk[b], dv[b] = dk32.transpose(0, 1), dv32.transpose(0, 1)
    o = _to_layout(c, o)
    if not train:
        return o, lse
    return o, lse, _to_layout(c, dq), _to_layout(c, dk), _to_layout(c, dv)


def _plain_paged(c, st):
    hq, hkv, d, page = c["hq"], c["hkv"], c["d"], c["page"]
    g = hq // hkv
    kp, vp = st["k_pages"].view(-1, hkv, d), st["v_pages"].view(-1, hkv, d)
    o = torch.empty_like(st["q"])
    lse = torch.empty((hq, len(o)), device="cuda")
    at = 0
    for b, (length, new) in enumerate(st["seqs"]):
        if not new:
            continue
        pos = torch.arange(length, device="cuda")
        slot = st["table"][b].long()[pos // page] * page + pos % page
        kp[slot[length - new:]] = st["k"][at:at + new]
        vp[slot[length - new:]] = st["v"][at:at + new]
        rows = max(1, (1 << 27) // (hq * length))
        for i0 in range(0, new, rows):
            i1 = min(new, i0 + rows)
            p1 = length - new + i1  # keys [p0, p1) of the sequence are seen
            p0 = max(0, p1 - (i1 - i0) - c["window"] + 1) if c["window"] else 0
            k = kp[slot[p0:p1]].transpose(0, 1).float()
            v = vp[slot[p0:p1]].transpose(0, 1).float()
            q = st["q"][at + i0:at + i1].float().transpose(0, 1).reshape(hkv, g * (i1 - i0), d)
            x = (q @ k.transpose(1, 2)).mul_(1.0 / math.sqrt(d)).view(hq, i1 - i0, p1 - p0)
            i = torch.arange(p1 - (i1 - i0), p1, device="cuda")[:, None]
            j = pos[p0:p1]
            see = j <= i
            if c["window"]:
                see &= j > i - c["window"]
            p, lse[:, at + i0:at + i1], _ = _plain_rows(x, see, c["cap"])
            o[at + i0:at + i1] = (p.view(hkv, -1, p1 - p0) @ v).view(hq, i1 - i0, d).transpose(0, 1)
        at += new
    return o, lse, st["k_pages"], st["v_pages"]


# --------------------------------------------------------------------- work
def work(case):
    c = case
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    if c["op"] == "mask":
        b, s = c["batch"], c["seqlen"]
        tok = b * s
        r = _ranges(c).long()
        pairs = hq * int((r[..., 1] - r[..., 0]).clamp(min=0).sum())
        place = 0 if c["see"] == "causal" and not (c["doc"] or c["pad"] or c["window"]) else 8 * tok
        qkv = (hq + 2 * hkv) * d
        if c["kind"] == "fwd":  # Q, K, V and the ranges in, O and LSE out; two products
            return {"bytes": 2 * (qkv + hq * d) * tok + 4 * hq * tok + place, "flops": 4 * d * pairs}
        # Q, K, V, dO and the ranges in, O, LSE, dQ, dK, dV out; two products and five
        return {"bytes": 2 * (2 * qkv + 2 * hq * d) * tok + 4 * hq * tok + place, "flops": 14 * d * pairs}
    pairs = kv = tok = 0
    for length, new in _sequences(c):
        tok += new
        for i in range(length - new, length):
            pairs += min(i + 1, c["window"]) if c["window"] else i + 1
        if new:
            old = length - new
            kv += min(old, c["window"] - 1) if c["window"] else old
    # the cached keys and values, the new tokens' Q, K, V in; K and V into the pages, O and LSE out
    return {"bytes": 4 * hkv * d * kv + 2 * tok * (2 * hq + 4 * hkv) * d + 4 * hq * tok, "flops": 4 * d * hq * pairs}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    return _exact_mask(case, st) if case["op"] == "mask" else _exact_paged(case, st)


def _exact_head(c, q, k, v, see):
    """Attention of one head in 64 bits; a row that sees nothing is 0, its LSE -inf."""
    x = q @ k.T / math.sqrt(c["d"])
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    w = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(w, -1)
    some = see.any(-1, keepdim=True)
    return torch.softmax(torch.where(some, w, 0.0), -1) * some @ v, lse


def _exact_mask(c, st):
    b_, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    train = c["kind"] == "train"
    nat = {n: _from_layout(c, st[n]) for n in ("q", "k", "v", "do") if n in st}
    f64 = {"dtype": torch.float64, "device": "cuda"}
    o, lse = torch.zeros((b_, s, hq, d), **f64), torch.full((b_, hq, s), -math.inf, **f64)
    if train:
        dq = torch.zeros_like(o)
        dk, dv = torch.zeros((b_, s, hkv, d), **f64), torch.zeros((b_, s, hkv, d), **f64)
    step = max(1, min(s, (1 << 25) // s))
    for b in range(b_):
        for i0 in range(0, s, step):
            rows = slice(i0, min(s, i0 + step))
            lo, hi = st["host_range"][b, rows].unbind(-1)
            live = lo < hi
            if not bool(live.any()):
                continue
            keys = slice(int(lo[live].min()), int(hi[live].max()))
            j = torch.arange(keys.start, keys.stop, device="cuda")
            lo, hi = lo.cuda()[:, None], hi.cuda()[:, None]
            see = ~((j < lo) | (j >= hi))
            for h in range(hq):
                kv = h * hkv // hq
                t = [nat["q"][b, rows, h].double(), nat["k"][b, keys, kv].double(), nat["v"][b, keys, kv].double()]
                if train:
                    for u in t:
                        u.requires_grad_(True)
                out, l = _exact_head(c, *t, see)
                o[b, rows, h] = out.detach()
                lse[b, h, rows] = l.detach()
                if train:
                    gq, gk, gv = torch.autograd.grad(out, t, nat["do"][b, rows, h].double())
                    dq[b, rows, h] = gq
                    dk[b, keys, kv] += gk
                    dv[b, keys, kv] += gv
    if not train:
        return _to_layout(c, o), lse
    return _to_layout(c, o), lse, _to_layout(c, dq), _to_layout(c, dk), _to_layout(c, dv)


def _exact_paged(c, st):
    hq, hkv, page = c["hq"], c["hkv"], c["page"]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    o = torch.empty_like(q)
    lse = torch.empty((hq, len(q)), dtype=torch.float64, device="cuda")
    at = 0
    for b, (length, new) in enumerate(st["seqs"]):
        if not new:
            continue
        pages = st["table"][b, :-(-length // page)].tolist()
        for x, y in ((kp, k), (vp, v)):
            for i in range(new):
                p = length - new + i
                x[pages[p // page], p % page] = y[at + i]
        ks = torch.cat([kp[p] for p in pages])[:length]
        vs = torch.cat([vp[p] for p in pages])[:length]
        step = max(1, (1 << 25) // length)
        for i0 in range(0, new, step):
            rows = slice(at + i0, at + min(new, i0 + step))
            back = (torch.arange(rows.start - at, rows.stop - at, device="cuda") + length - new)[:, None] - \
                torch.arange(length, device="cuda")
            see = back >= 0
            if c["window"]:
                see = see & (back < c["window"])
            for h in range(hq):
                kv = h * hkv // hq
                o[rows, h], lse[h, rows] = _exact_head(c, q[rows, h], ks[:, kv], vs[:, kv], see)
        at += new
    return o, lse, kp, vp
