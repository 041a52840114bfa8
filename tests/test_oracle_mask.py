"""The masked attention's float64 oracle against finite differences and closed
forms."""
import numpy as np
import pytest

from oracle import attention, mask


def _small(seed, s=9, hq=4, hkv=2, d=6):
    r = np.random.default_rng(seed)
    return tuple(r.standard_normal((s, h, d)) for h in (hq, hkv, hkv, hq))


RANGES = np.array([[0, 3], [0, 3], [1, 3], [5, 5], [3, 9], [-4, 20], [8, 9], [6, 2], [0, 9]])


@pytest.mark.parametrize("cap", [0.0, 0.7, 30.0])
@pytest.mark.parametrize("causal", [True, False])
def test_gradients_are_the_differences(causal, cap):
    q, k, v, do = _small(1)
    see = mask.sees(RANGES, 9, causal)
    f = lambda q, k, v: (mask.forward_backward(q, k, v, None, see, 0.4, cap)["o"] * do).sum()
    out = mask.forward_backward(q, k, v, do, see, 0.4, cap)
    args, r, h = [q, k, v], np.random.default_rng(2), 1e-5
    for i, name in enumerate(("dq", "dk", "dv")):
        for _ in range(6):
            u = r.standard_normal(args[i].shape)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * u, args[i] - h * u
            # central difference: error h^2 times third derivatives (order 1e2 here) plus 1e-16 / h
            assert abs((f(*up) - f(*down)) / (2 * h) - (out[name] * u).sum()) < 1e-7, name


@pytest.mark.parametrize("causal", [True, False])
def test_whole_ranges_change_nothing(causal):
    q, k, v, _ = _small(3)
    see = mask.sees(np.tile([0, 9], (9, 1)), 9, causal)
    out = mask.forward_backward(q, k, v, None, see, 0.4)
    o, lse = attention.attention_forward(q, k, v, scale=0.4, causal=causal)
    np.testing.assert_allclose(out["o"], o, atol=1e-12)
    np.testing.assert_allclose(out["lse"], lse, atol=1e-12)
    # a cap far above the scores neither: cap tanh(x / cap) = x - x^3 / (3 cap^2)
    far = mask.forward_backward(q, k, v, None, see, 0.4, 1e6)
    np.testing.assert_allclose(far["o"], o, atol=1e-9)


def test_rows_that_see_nothing_and_keys_not_seen():
    q, k, v, do = _small(4)
    see = mask.sees(RANGES, 9, True)
    out = mask.forward_backward(q, k, v, do, see, 0.4)
    for i in (3, 7):
        assert np.all(out["o"][i] == 0) and np.all(np.isneginf(out["lse"][:, i])) and np.all(out["dq"][i] == 0)
    one = mask.sees(np.tile([2, 3], (9, 1)), 9, False)
    k[4], v[5] = np.nan, np.inf     # keys that nobody sees
    out = mask.forward_backward(q, k, v, do, one, 0.4)
    np.testing.assert_allclose(out["o"][:, 1], v[np.full(9, 2), 0], atol=1e-12)
    assert np.all(out["dk"][4] == 0) and np.all(out["dv"][5] == 0)
