"""Plain float64 attention with a bucketed relative position bias.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

logit_ij = scale q_i.k_j + table[bucket(i - j), head]; softmax over the keys a
query sees (all, or j <= i); with dP = dO V^T, D_i = dO_i . O_i and
dS = P (dP - D): dtable[t, head] = sum of dS_ij over bucket(i - j) = t, the other
gradients as in ``oracle.attention``.  A logit of -inf has weight 0; a query all
of whose logits are -inf gets O = 0, LSE = -inf and no gradient.  bucket(n) =
bucket_of[number of bounds <= n].

Layouts: q [S, Hq, d], k and v [S, Hkv, d], table [buckets, Hq].
"""
import numpy as np


def buckets_of_distance(n, bounds, bucket_of):
    return np.asarray(bucket_of)[np.searchsorted(np.asarray(bounds, dtype=np.int64), n, side="right")]


def forward_backward(q, k, v, do, table, bounds, bucket_of, scale, causal, terms=False):
    """dict of o, lse and, with ``do``, dq, dk, dv, dtable.  ``terms`` adds what
    error bounds are made of: the same sums over absolute values."""
    q, k, v, table = (np.asarray(t, dtype=np.float64) for t in (q, k, v, table))
    s, hq, d = q.shape
    g = hq // k.shape[1]
    n = np.arange(s)[:, None] - np.arange(s)[None, :]
    bucket = buckets_of_distance(n, bounds, bucket_of)
    out = {"o": np.zeros((s, hq, d)), "lse": np.full((hq, s), -np.inf)}
    if do is not None:
        do = np.asarray(do, dtype=np.float64)
        out |= {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v), "dtable": np.zeros_like(table)}
    if terms:
        out |= {"abs_" + x: np.zeros_like(out[x]) for x in out if x != "lse"} | {"logit": np.zeros((hq, s))}
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        x = scale * (q[:, h] @ kk.T) + table[bucket, h]
        if causal:
            x[n < 0] = -np.inf
        m = x.max(axis=1, keepdims=True)
        m[~np.isfinite(m)] = 0.0
        e = np.exp(x - m)
        l = e.sum(axis=1, keepdims=True)
        some = l > 0
        p = np.divide(e, l, out=np.zeros_like(e), where=some)
        o = p @ vv
        out["o"][:, h] = o
        with np.errstate(divide="ignore"):
            out["lse"][h] = np.where(some, m + np.log(l), -np.inf)[:, 0]
        if terms:
            out["abs_o"][:, h] = p @ np.abs(vv)
            out["logit"][h] = scale * np.linalg.norm(q[:, h], axis=1) * np.linalg.norm(kk, axis=1).max() + \
                np.abs(np.where(np.isfinite(table[:, h]), table[:, h], 0)).max()
        if do is None:
            continue
        dp = do[:, h] @ vv.T
        ds = p * (dp - (do[:, h] * o).sum(axis=1, keepdims=True))
        out["dq"][:, h] = scale * (ds @ kk)
        out["dk"][:, h // g] += scale * (ds.T @ q[:, h])
        out["dv"][:, h // g] += p.T @ do[:, h]
        np.add.at(out["dtable"][:, h], bucket.ravel(), ds.ravel())
        if terms:
            # |dS| with every part of dP - D taken as an absolute value
            a = p * (np.abs(do[:, h]) @ np.abs(vv).T + (np.abs(do[:, h]) * out["abs_o"][:, h]).sum(axis=1, keepdims=True))
            out["abs_dq"][:, h] = scale * (a @ np.abs(kk))
            out["abs_dk"][:, h // g] += scale * (a.T @ np.abs(q[:, h]))
            out["abs_dv"][:, h // g] += p.T @ np.abs(do[:, h])
            np.add.at(out["abs_dtable"][:, h], bucket.ravel(), a.ravel())
    return out
