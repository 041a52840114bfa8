"""The relative bias's float64 oracle against finite differences and closed
forms."""
import numpy as np
import pytest

from oracle import attention, bias


def _small(seed, s=9, hq=4, hkv=2, d=6, buckets=5):
    r = np.random.default_rng(seed)
    return (r.standard_normal((s, hq, d)), r.standard_normal((s, hkv, d)), r.standard_normal((s, hkv, d)),
            r.standard_normal((s, hq, d)), r.standard_normal((buckets, hq)))


BOUNDS, BUCKET_OF = [-3, 0, 1, 2, 5], [4, 3, 0, 1, 2, 4]


@pytest.mark.parametrize("causal", [True, False])
def test_bias_gradients_are_the_differences(causal):
    q, k, v, do, table = _small(1)
    f = lambda q, k, v, t: (bias.forward_backward(q, k, v, None, t, BOUNDS, BUCKET_OF, 0.4, causal)["o"] * do).sum()
    out = bias.forward_backward(q, k, v, do, table, BOUNDS, BUCKET_OF, 0.4, causal)
    args, r, h = [q, k, v, table], np.random.default_rng(2), 1e-5
    for i, name in enumerate(("dq", "dk", "dv", "dtable")):
        for _ in range(6):
            u = r.standard_normal(args[i].shape)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * u, args[i] - h * u
            # central difference: error h^2 times third derivatives (order 1e2 here) plus 1e-16 / h
            assert abs((f(*up) - f(*down)) / (2 * h) - (out[name] * u).sum()) < 1e-7, name


@pytest.mark.parametrize("causal", [True, False])
def test_one_value_everywhere_changes_nothing(causal):
    q, k, v, do, table = _small(3)
    out = bias.forward_backward(q, k, v, do, np.full_like(table, 0.7), BOUNDS, BUCKET_OF, 0.4, causal)
    o, lse = attention.attention_forward(q, k, v, scale=0.4, causal=causal)
    np.testing.assert_allclose(out["o"], o, atol=1e-12)
    np.testing.assert_allclose(out["lse"], lse + 0.7, atol=1e-12)
    # softmax does not change with a shift of a row's logits
    np.testing.assert_allclose(out["dtable"].sum(axis=0), 0, atol=1e-12)


def test_bias_of_minus_infinity_masks():
    q, k, v, do, table = _small(4)
    table[0] = -np.inf                       # distance 0
    out = bias.forward_backward(q, k, v, do, table, [1, 2, 3, 4], [0, 1, 2, 3, 4], 0.4, True)
    assert np.all(out["o"][0] == 0) and np.all(np.isneginf(out["lse"][:, 0]))   # query 0 only has itself
    assert np.all(out["dq"][0] == 0) and np.all(out["dtable"][0] == 0)
    assert all(np.all(np.isfinite(out[n])) for n in ("o", "dq", "dk", "dv", "dtable"))
