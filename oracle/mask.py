"""Plain float64 attention over a range of keys for every query, with capped scores.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

logit_ij = scale q_i.k_j, or cap tanh(scale q_i.k_j / cap) with cap > 0; softmax
over the keys begin_i <= j < end_i (and j <= i with ``causal``); with
dP = dO V^T, D_i = dO_i . O_i and dS = P (dP - D) (1 - (logit / cap)^2) the other
gradients as in ``oracle.attention``.  A query that sees no key gets O = 0,
LSE = -inf and no gradient.  Keys that a query does not see take no part in any
sum, whatever they hold.

Layouts: q [S, Hq, d], k and v [keys, Hkv, d], ranges [S, 2].
"""
import numpy as np


def sees(ranges, keys, causal, first=0):
    """[S, keys] truth values; query i stands at position first + i."""
    r = np.asarray(ranges, dtype=np.int64)
    j = np.arange(keys)[None, :]
    see = (j >= r[:, :1]) & (j < r[:, 1:])
    if causal:
        see &= j <= first + np.arange(len(r))[:, None]
    return see


def forward_backward(q, k, v, do, see, scale, cap=0.0, terms=False):
    """dict of o, lse and, with ``do``, dq, dk, dv.  ``terms`` adds what error
    bounds are made of: the same sums over absolute values, with (abs_) and
    without (flat_) the cap's derivative."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    s, hq, d = q.shape
    g = hq // k.shape[1]
    out = {"o": np.zeros((s, hq, d)), "lse": np.full((hq, s), -np.inf)}
    if do is not None:
        do = np.asarray(do, dtype=np.float64)
        out |= {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    if terms:
        names = [x for x in out if x != "lse"]
        out |= {"abs_" + x: np.zeros_like(out[x]) for x in names} | {"flat_" + x: np.zeros_like(out[x]) for x in names}
        out["logit"] = np.zeros((hq, s))
    some = see.any(axis=1, keepdims=True)
    used, live = see.any(axis=0), some[:, 0]
    # what takes no part is 0, so that 0 times it is 0
    q = np.where(live[:, None, None], q, 0)
    k, v = (np.where(used[:, None, None], t, 0) for t in (k, v))
    if do is not None:
        do = np.where(live[:, None, None], do, 0)
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        x = scale * (q[:, h] @ kk.T)
        slope = 1.0
        if cap > 0:
            t = np.tanh(x / cap)
            x, slope = cap * t, 1 - t * t
        x = np.where(see, x, -np.inf)
        m = np.where(some, x.max(axis=1, keepdims=True, initial=-np.inf), 0)
        e = np.exp(x - m)
        l = e.sum(axis=1, keepdims=True)
        p = e / np.where(some, l, 1)
        o = p @ vv
        out["o"][:, h] = o
        out["lse"][h] = np.where(some, m + np.log(np.where(some, l, 1)), -np.inf)[:, 0]
        if terms:
            out["abs_o"][:, h] = p @ np.abs(vv)
            out["logit"][h] = scale * np.linalg.norm(q[:, h], axis=1) * np.linalg.norm(kk, axis=1).max(initial=0)
        if do is None:
            continue
        dp = do[:, h] @ vv.T
        ds = p * (dp - (do[:, h] * o).sum(axis=1, keepdims=True)) * slope
        out["dq"][:, h] = scale * (ds @ kk)
        out["dk"][:, h // g] += scale * (ds.T @ q[:, h])
        out["dv"][:, h // g] += p.T @ do[:, h]
        if terms:
            flat = p * (np.abs(do[:, h]) @ np.abs(vv).T +
                        (np.abs(do[:, h]) * out["abs_o"][:, h]).sum(axis=1, keepdims=True))
            for name, a in (("abs_", flat * slope), ("flat_", flat)):
                out[name + "dq"][:, h] = scale * (a @ np.abs(kk))
                out[name + "dk"][:, h // g] += scale * (a.T @ np.abs(q[:, h]))
                out[name + "dv"][:, h // g] += p.T @ np.abs(do[:, h])
    return out
