"""Workloads of the positional operators around the ring attention.

Two operators, forward and backward:

* ``qk``: the RMS norm of every query and key head, the rotation of (a part
  of) each head by its token's position, and the layout the attention reads
  (natural, or every emulated rank's layout), out of one fused projection.
* ``bias``: ring attention whose scaled scores get a learned bias that depends
  on the bucket of the distance query - key, with the gradient of the bias.

A case is a dict of plain values.  ``prepare`` makes its inputs, ``run`` makes
one pass, in elementary torch operations or (``own``) through the package.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- the cases
def _qk(name, kind, batch, seqlen, hq, hkv, d, hp=1, cp=1, zigzag=True, rank_major=False, rot=None, interleaved=False,
        base=500000.0, packed=False, pos=0):
    return {"name": name, "op": "qk", "kind": kind, "batch": batch, "seqlen": seqlen, "hq": hq, "hkv": hkv, "d": d,
            "hp": hp, "cp": cp, "zigzag": zigzag, "rank_major": rank_major, "rot": d if rot is None else rot,
            "interleaved": interleaved, "base": base, "packed": packed, "pos": pos}


def _bias(name, kind, batch, seqlen, hq, hkv, d, hp=1, cp=1, zigzag=True, rank_major=False, causal=True, buckets=32,
          max_distance=128, stepwise=False):
    return {"name": name, "op": "bias", "kind": kind, "batch": batch, "seqlen": seqlen, "hq": hq, "hkv": hkv, "d": d,
            "hp": hp, "cp": cp, "zigzag": zigzag, "rank_major": rank_major, "causal": causal, "buckets": buckets,
            "max_distance": max_distance, "stepwise": stepwise}


def listed():
    return [
        # one new token of one sequence, far into its context
        _qk("qk-token", "fwd", 1, 1, 32, 8, 128, zigzag=False, pos=40000),
        # one new token of each of 61 sequences, each at its own position
        _qk("qk-tokens-b61", "fwd", 61, 1, 64, 8, 128, zigzag=False, packed=True, pos=131072),
        # the 8B layer at 32K tokens, written straight into the ranks' layout
        _qk("qk-8b-s32k", "fwd", 1, 32768, 32, 8, 128, hp=4, cp=8, rank_major=True),
        # packed documents of an odd length, part of the head rotated in adjacent pairs
        _qk("qk-odd-bwd", "bwd", 3, 1001, 10, 5, 64, zigzag=False, rot=32, interleaved=True, base=10000.0, packed=True),
        # the 8B layer's gradient at 128K tokens, read from the ranks' layout
        _qk("qk-8b-s128k-bwd", "bwd", 1, 131072, 32, 8, 128, hp=8, cp=16, rank_major=True),
        # a short prompt through a small layer
        _bias("bias-short", "fwd", 1, 100, 4, 2, 64, zigzag=False),
        # an encoder: every key, distances of both signs
        _bias("bias-encoder-s4k", "fwd", 2, 4096, 16, 16, 128, zigzag=False, causal=False),
        # the 8B layer at 32K tokens, prefill on the ranks' layout
        _bias("bias-8b-s32k", "fwd", 1, 32768, 32, 8, 128, hp=4, cp=8, rank_major=True),
        # a training step of the tiny layer
        _bias("bias-tiny-s1k-train", "train", 1, 1024, 4, 2, 64, hp=2, cp=4),
        # a ragged training step, every key, blocks that are no multiple of a tile
        _bias("bias-odd-train", "train", 2, 1990, 6, 3, 64, cp=5, causal=False),
        # a training step of the 8B layer, buckets that reach far into the context
        _bias("bias-8b-s16k-train", "train", 1, 16384, 32, 8, 128, hp=8, cp=16, buckets=64, max_distance=8192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    hkv = rng.randint(1, 8)
    hq = hkv * rng.randint(1, 8)
    cp = rng.choice([1, 1, 2, 3, 4, 8])
    hp = rng.choice([p for p in (1, 1, 2, 4) if hkv % p == 0])
    zigzag = rng.random() < 0.7
    unit = (2 * cp if zigzag else cp) * hp  # the sequence length is a multiple of this
    batch = rng.randint(1, 3)
    rank_major = rng.random() < 0.5
    if rng.random() < 0.5:
        if rng.random() < 0.3:  # new tokens
            return _qk("", rng.choice(["fwd", "fwd", "bwd"]), _log_int(rng, 1, 512), rng.randint(1, 4), hq, hkv, d,
                       zigzag=False, packed=rng.random() < 0.5, pos=_log_int(rng, 1, 1 << 20))
        most = 131072 * 48 * 128 // (batch * (hq + 2 * hkv) * d)
        s = unit * max(1, _log_int(rng, 17, min(most, 131072)) // unit)
        return _qk("", rng.choice(["fwd", "bwd"]), batch, s, hq, hkv, d, hp, cp, zigzag, rank_major,
                   rng.choice([d, d, d // 2, 16]), rng.random() < 0.3, rng.choice([10000.0, 500000.0]),
                   rng.random() < 0.5, rng.choice([0, 0, 4096]))
    train = rng.random() < 0.6
    causal = rng.random() < 0.7
    # scores of the largest listed passes: half of 32768^2 (forward), of 16384^2 (training), 32 heads of 128
    most = (16384 if train else 32768) ** 2 * 32 * 128 // 2
    top = math.sqrt(most * (2 if causal else 1) / (batch * hq * d))
    s = unit * max(1, _log_int(rng, 20, min(top, 65536)) // unit)
    return _bias("", "train" if train else "fwd", batch, s, hq, hkv, d, hp, cp, zigzag, rank_major, causal,
                 rng.choice([8, 32, 64]), _log_int(rng, 64, 16384), rng.random() < 0.2)


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


def _buckets(c):
    """(bounds, bucket_of): distance n lies in interval #{bounds <= n}, interval
    i in bucket bucket_of[i].  Half of a direction's buckets hold one distance
    each, the rest grow by a constant factor up to max_distance."""
    n = c["buckets"] if c["causal"] else c["buckets"] // 2
    e = n // 2
    m = max(c["max_distance"], e + 1)
    starts = list(range(1, e + 1))  # first distance of buckets 1, 2, ...
    for t in range(1, n - e):
        x = max(1, int(e * (m / e) ** (t / (n - e))) - 2)
        while x ** (n - e) * e ** t < m ** t * e ** (n - e):
            x += 1
        starts.append(x)
    ids = {}
    for i, x in enumerate(starts):
        ids[x] = i + 1  # where two buckets start at one distance, the later one has it
    pos = sorted(ids)
    bounds, of = list(pos), [0] + [ids[x] for x in pos]
    if not c["causal"]:  # distances below zero: buckets n, n + 1, ...
        bounds = [1 - x for x in reversed(pos)] + bounds
        of = [n + ids[x] for x in reversed(pos)] + of
    return bounds, of


# ------------------------------------------------------------------ prepare
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    st = {"case": c}
    if c["op"] == "qk":
        # the output of the fused projection: Q, K, V side by side for each token
        st["x"] = (_normal(g, b, s, (hq + 2 * hkv) * d) * 1.5).to(torch.bfloat16)
        st["wq"] = 1 + 0.2 * _normal(g, d)
        st["wk"] = 1 + 0.2 * _normal(g, d)
        st["positions"] = None
        if c["packed"]:  # documents (or sequences) that start anywhere
            start = torch.randint(0, max(1, c["pos"]) + 1, (b, 1), generator=g, device="cuda")
            cut = torch.randint(0, s + 1, (b, 1), generator=g, device="cuda")
            t = torch.arange(s, device="cuda").expand(b, s)
            st["positions"] = torch.where(t < cut, start + t, t - cut).contiguous()
        if c["kind"] == "bwd":
            for n, h in (("dq", hq), ("dk", hkv), ("dv", hkv)):
                st[n] = _to_layout(c, _normal(g, b, s, h, d).to(torch.bfloat16))
        if own:
            from head_context_attention_gb300 import inputs, ops
            st["w"] = inputs.Workload("qk", s, hq, hkv, d, c["hp"], c["cp"], c["cp"], 1, True, batch=b,
                                      placement=1 if c["zigzag"] else 0)
            st["opts"] = ops.make_qk_opts(d, eps=EPS, rot_dim=c["rot"], base=c["base"], interleaved=c["interleaved"])
        return st
    for n, h in (("q", hq), ("k", hkv), ("v", hkv), ("do", hq)):
        if n != "do" or c["kind"] == "train":
            st[n] = _to_layout(c, _normal(g, b, s, h, d).to(torch.bfloat16))
    st["table"] = _normal(g, c["buckets"], hq).to(torch.bfloat16)
    st["bounds"], st["bucket_of"] = _buckets(c)
    if own:
        from head_context_attention_gb300 import inputs, ops
        st["w"] = inputs.Workload("bias", s, hq, hkv, d, c["hp"], c["cp"], c["cp"], 1, c["kind"] == "train", batch=b,
                                  placement=1 if c["zigzag"] else 0, causal=c["causal"])
        st["buckets"] = ops.RelBuckets(c["buckets"], st["bounds"], st["bucket_of"])
    return st


# ---------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if own:
        return _own_qk(c, state) if c["op"] == "qk" else _own_bias(c, state)
    return _plain_qk(c, state) if c["op"] == "qk" else _plain_bias(c, state)


def _split(c, x):
    """Q, K, V of a fused projection, [B, S, H, d] views."""
    b, s, _ = x.shape
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    q, k, v = x.split([hq * d, hkv * d, hkv * d], dim=2)
    return q.unflatten(2, (hq, d)), k.unflatten(2, (hkv, d)), v.unflatten(2, (hkv, d))


def _own_qk(c, st):
    from head_context_attention_gb300 import ops
    q, k, v = _split(c, st["x"])
    layout = ops.LAYOUT_RANK_MAJOR if c["rank_major"] else ops.LAYOUT_NATURAL
    place = {"wq": st["wq"], "wk": st["wk"], "positions": st["positions"], "layout": layout,
             "pos_begin": 0 if c["packed"] else c["pos"]}
    if c["kind"] == "fwd":
        return ops.qk_norm_rope(st["w"], st["opts"], q, k, v, **place)
    dx = torch.empty_like(st["x"])
    _, _, _, dwq, dwk = ops.qk_norm_rope_bwd(st["w"], st["opts"], q, k, st["dq"], st["dk"], st["dv"],
                                             into=_split(c, dx), **place)
    return dx, dwq, dwk


def _own_bias(c, st):
    from head_context_attention_gb300 import ops
    how = {"mode": ops.MODE_STEPWISE if c["stepwise"] else ops.MODE_FUSED,
           "layout": ops.LAYOUT_RANK_MAJOR if c["rank_major"] else ops.LAYOUT_NATURAL}
    w, q, k, v, table, buckets = (st[n] for n in ("w", "q", "k", "v", "table", "buckets"))
    train = c["kind"] == "train"
    o, lse, o_res = ops.attn_bias_fwd(w, q, k, v, table, buckets, res=train, **how)
    if not train:
        return o, lse
    return (o, lse) + ops.attn_bias_bwd(w, q, k, v, o, lse, st["do"], table, buckets, o_res=o_res, **how)


# -------------------------------------------------------------- plain forms
def _cos_sin(c, positions):
    """cos, sin [B, S, 1, rot / 2] in fp32 of angles formed in 64 bits."""
    r = c["rot"]
    inv = c["base"] ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if positions is None:
        positions = (c["pos"] + torch.arange(c["seqlen"], device="cuda")).expand(c["batch"], -1)
    a = positions.double()[:, :, None, None] * inv
    return a.cos().float(), a.sin().float()


def _rotate(c, x, cos, sin):
    """The first rot elements of every head, in pairs, by (cos, sin)."""
    r = c["rot"]
    if c["interleaved"]:
        p = x[..., :r].unflatten(-1, (r // 2, 2))
        a, b = p[..., 0], p[..., 1]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((y, x[..., r:]), dim=-1)


def _plain_qk(c, st):
    q, k, v = _split(c, st["x"])
    cos, sin = _cos_sin(c, st["positions"])
    if c["kind"] == "fwd":
        def one(x, w):
            x = x.float()
            y = x * ((x * x).mean(-1, keepdim=True) + EPS).rsqrt() * w
            return _to_layout(c, _rotate(c, y, cos, sin).to(torch.bfloat16))
        return one(q, st["wq"]), one(k, st["wk"]), _to_layout(c, v).contiguous()
    dx = torch.empty_like(st["x"])
    dq, dk, dv = _split(c, dx)

    def grad(x, w, dy, into):
        x = x.float()
        r = ((x * x).mean(-1, keepdim=True) + EPS).rsqrt()
        x = x * r
        dy = _rotate(c, _from_layout(c, dy).float(), cos, -sin)
        dw = (dy * x).sum((0, 1), dtype=torch.float64).sum(0).float()
        dy = dy * w
        into.copy_(r * (dy - x * (dy * x).mean(-1, keepdim=True)))
        return dw
    dwq = grad(q, st["wq"], st["dq"], dq)
    dwk = grad(k, st["wk"], st["dk"], dk)
    dv.copy_(_from_layout(c, st["dv"]))
    return dx, dwq, dwk


def _bias_of_distance(c, st):
    """Bias of every head at distances -(S-1) .. S-1, [hq, 2S-1], and their buckets."""
    n = torch.arange(1 - c["seqlen"], c["seqlen"], device="cuda")
    bounds = torch.tensor(st["bounds"], device="cuda")
    ids = torch.tensor(st["bucket_of"], device="cuda")[(n[:, None] >= bounds).sum(1)]
    return st["table"].float()[ids].t().contiguous(), ids


def _plain_bias(c, st):
    train = c["kind"] == "train"
    b_, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    scale = 1.0 / math.sqrt(d)
    lut, ids = _bias_of_distance(c, st)
    slide = lut.flip(1).unfold(1, s, 1)  # [hq, S, S]: row S-1-i of a head is the bias of query i over all keys
    names = ("q", "k", "v", "do") if train else ("q", "k", "v")
    nat = {n: _from_layout(c, st[n]) for n in names}
    o = torch.empty((b_, s, hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b_, hq, s), device="cuda")
    if train:
        dq = torch.empty_like(o)
        dk, dv = torch.empty_like(nat["k"]), torch.empty_like(nat["v"])
        ddist = torch.zeros((hq, 2 * s - 1), dtype=torch.float64, device="cuda")
    rows = max(1, min(s, (1 << 28) // (hq * s)))
    for b in range(b_):
        k = nat["k"][b].transpose(0, 1).float()  # [hkv, S, d]
        v = nat["v"][b].transpose(0, 1).float()
        if train:
            dk32, dv32 = torch.zeros_like(k), torch.zeros_like(v)
        for i0 in range(0, s, rows):
            i1 = min(s, i0 + rows)
            n, keys = i1 - i0, i1 if c["causal"] else s
            q = nat["q"][b, i0:i1].float().transpose(0, 1).reshape(hkv, g * n, d)
            kc, vc = k[:, :keys], v[:, :keys]
            x = (q @ kc.transpose(1, 2)).mul_(scale).view(hq, n, keys)
            i = torch.arange(i0, i1, device="cuda")
            x += slide[:, s - 1 - i, :keys]
            if c["causal"]:
                x.masked_fill_(torch.arange(keys, device="cuda") > i[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            p = x.sub_(top).exp_()
            l = p.sum(-1, keepdim=True)
            p = p.div_(l).view(hkv, g * n, keys)
            o32 = p @ vc
            o[b, i0:i1] = o32.view(hq, n, d).transpose(0, 1)
            lse[b, :, i0:i1] = (top + l.log()).squeeze(-1)
            if not train:
                continue
            do = nat["do"][b, i0:i1].float().transpose(0, 1).reshape(hkv, g * n, d)
            dv32[:, :keys] += p.transpose(1, 2) @ do
            ds = do @ vc.transpose(1, 2)
            ds = ds.sub_((do * o32).sum(-1, keepdim=True)).mul_(p)
            dq[b, i0:i1] = (ds @ kc).mul_(scale).view(hq, n, d).transpose(0, 1)
            dk32[:, :keys] += (ds.transpose(1, 2) @ q).mul_(scale)
            # sums over the diagonals: rows of keys in falling order, each shifted one further, summed down
            f = torch.nn.functional.pad(ds.view(hq, n, keys).flip(2), (0, n)).flatten(1)
            f = f[:, :n * (keys + n - 1)].view(hq, n, keys + n - 1).sum(1, dtype=torch.float64)
            lo = i0 - (keys - 1) + s - 1  # place of distance i0 - (keys - 1)
            ddist[:, lo:lo + keys + n - 1] += f
        if train:
            dk[b], dv[b] = dk32.transpose(0, 1), dv32.transpose(0, 1)
    o = _to_layout(c, o)
    if not train:
        return o, lse
    dtable = torch.zeros((c["buckets"], hq), dtype=torch.float64, device="cuda").index_add_(0, ids, ddist.t())
    return o, lse, _to_layout(c, dq), _to_layout(c, dk), _to_layout(c, dv), dtable.to(torch.bfloat16)


# --------------------------------------------------------------------- work
def work(case):
    c = case
    b, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    tok = b * s
    qkv = (hq + 2 * hkv) * d
    if c["op"] == "qk":
        pos = 8 * tok if c["packed"] else 0
        if c["kind"] == "fwd":  # the projection in, Q, K, V out; norm 5, rotation 3 per element
            return {"bytes": 2 * 2 * qkv * tok + pos + 2 * 4 * d, "flops": 8 * (hq + hkv) * d * tok}
        # Q, K and three gradients in, three gradients and two weight gradients out
        return {"bytes": 2 * (qkv + (hq + hkv) * d + qkv) * tok + pos + 4 * 4 * d, "flops": 16 * (hq + hkv) * d * tok}
    pairs = b * hq * (s * (s + 1) // 2 if c["causal"] else s * s)
    table = 2 * c["buckets"] * hq
    if c["kind"] == "fwd":  # Q, K, V and the table in, O and LSE out; two products
        return {"bytes": 2 * (qkv + hq * d) * tok + 4 * hq * tok + table, "flops": 4 * d * pairs}
    # Q, K, V, dO and the table in, O, LSE, dQ, dK, dV and the table's gradient out; two products and five
    return {"bytes": 2 * (2 * qkv + 2 * hq * d) * tok + 4 * hq * tok + 2 * table, "flops": 14 * d * pairs}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    if case["op"] == "bias" and work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    return _exact_qk(case, st) if case["op"] == "qk" else _exact_bias(case, st)


def _exact_qk(c, st):
    """One chunk of tokens after the other; the pairs of a head as complex
    numbers, the gradients by differentiating the definition."""
    b, s, hq, hkv, d, r = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"], c["rot"]
    bwd = c["kind"] == "bwd"
    freq = torch.tensor([c["base"] ** (-2.0 * i / r) for i in range(r // 2)], dtype=torch.float64, device="cuda")
    if st["positions"] is None:
        place = torch.arange(c["pos"], c["pos"] + s, device="cuda").repeat(b, 1)
    else:
        place = st["positions"]

    def op(x, w, turn):
        y = x / torch.sqrt(x.square().sum(-1, keepdim=True) / d + EPS) * w
        head, rest = y[..., :r], y[..., r:]
        if c["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * turn
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(head[..., :r // 2], head[..., r // 2:]) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, rest), -1)

    x = st["x"]
    ws = [st["wq"].double(), st["wk"].double()]
    widths = [hq * d, hkv * d]
    if not bwd:
        outs = [torch.empty((b, s, h, d), dtype=torch.float64, device="cuda") for h in (hq, hkv)]
    else:
        dx = torch.empty(x.shape, dtype=torch.float64, device="cuda")
        dws = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in ws]
        dys = [_from_layout(c, st["dq"]), _from_layout(c, st["dk"])]
        dx[..., sum(widths):] = _from_layout(c, st["dv"]).reshape(b, s, hkv * d).double()
    step = max(1, (1 << 26) // (b * (hq + hkv) * d))
    for s0 in range(0, s, step):
        sl = slice(s0, min(s, s0 + step))
        ang = place[:, sl].double()[..., None] * freq
        turn = torch.polar(torch.ones_like(ang), ang)[:, :, None]
        at = 0
        for j, h in enumerate((hq, hkv)):
            xi = x[:, sl, at:at + h * d].double().unflatten(2, (h, d))
            at += h * d
            if not bwd:
                outs[j][:, sl] = op(xi, ws[j], turn)
                continue
            xi.requires_grad_(True)
            wi = ws[j].clone().requires_grad_(True)
            gx, gw = torch.autograd.grad(op(xi, wi, turn), (xi, wi), dys[j][:, sl].double())
            dx[:, sl, at - h * d:at] = gx.flatten(2)
            dws[j] += gw
    if bwd:
        return dx, dws[0], dws[1]
    v = x[..., sum(widths):].unflatten(2, (hkv, d)).double()
    return _to_layout(c, outs[0]), _to_layout(c, outs[1]), _to_layout(c, v)


def _exact_bias(c, st):
    """Softmax attention from its definition, some rows of one head at a time,
    its gradients by differentiating it."""
    b_, s, hq, hkv, d = c["batch"], c["seqlen"], c["hq"], c["hkv"], c["d"]
    train = c["kind"] == "train"
    nat = {n: _from_layout(c, st[n]) for n in ("q", "k", "v", "do") if n in st}
    f64 = {"dtype": torch.float64, "device": "cuda"}
    o, lse = torch.empty((b_, s, hq, d), **f64), torch.empty((b_, hq, s), **f64)
    table = st["table"].double()
    bounds = torch.tensor(st["bounds"], device="cuda")
    of = torch.tensor(st["bucket_of"], device="cuda")
    if train:
        dq, dtable = torch.empty_like(o), torch.zeros_like(table)
        dk, dv = torch.zeros((b_, s, hkv, d), **f64), torch.zeros((b_, s, hkv, d), **f64)
    j = torch.arange(s, device="cuda")
    step = max(1, min(s, (1 << 25) // s))
    for i0 in range(0, s, step):
        i = torch.arange(i0, min(s, i0 + step), device="cuda")
        keys = int(i[-1]) + 1 if c["causal"] else s
        bucket = of[torch.bucketize(i[:, None] - j[:keys], bounds, right=True)]
        seen = (j[:keys] <= i[:, None]) if c["causal"] else torch.ones((len(i), keys), dtype=torch.bool, device="cuda")
        for b in range(b_):
            for h in range(hq):
                kv = h * hkv // hq
                t = [nat["q"][b, i, h].double(), nat["k"][b, :keys, kv].double(), nat["v"][b, :keys, kv].double(),
                     table[:, h].clone()]
                if train:
                    for u in t:
                        u.requires_grad_(True)
                add = t[3][bucket].detach().requires_grad_(train)  # its gradient is summed by bucket below
                x = torch.where(seen, t[0] @ t[1].T / math.sqrt(d) + add, -math.inf)
                out = torch.softmax(x, -1) @ t[2]
                o[b, i, h] = out.detach()
                lse[b, h, i] = torch.logsumexp(x.detach(), -1)
                if train:
                    gq, gk, gv, ga = torch.autograd.grad(out, (*t[:3], add), nat["do"][b, i, h].double())
                    dq[b, i, h] = gq
                    dk[b, :keys, kv] += gk
                    dv[b, :keys, kv] += gv
                    dtable[:, h] += torch.bincount(bucket.flatten(), ga.flatten(), minlength=c["buckets"])
    if not train:
        return _to_layout(c, o), lse
    return _to_layout(c, o), lse, _to_layout(c, dq), _to_layout(c, dk), _to_layout(c, dv), dtable
