"""The norm-and-rotation float64 oracle against finite differences and
closed forms."""
import numpy as np
import pytest

from oracle import qk


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_gradients_are_the_differences(interleaved, norm):
    r = np.random.default_rng(5)
    x, w, dy = r.standard_normal((5, 3, 8)), r.standard_normal(8), r.standard_normal((5, 3, 8))
    m = qk.matrices([0, 1, 7, -3, 1000], 8, 6 if interleaved else 4, [1.0, 0.3, 0.01], interleaved, 1.25)
    f = lambda x, w: (qk.forward(x, w, m, 1e-3, norm, 0.5) * dy).sum()
    dx, dw = qk.backward(x, w, m, 1e-3, dy, norm, 0.5)
    h = 1e-5
    for _ in range(8):
        u = r.standard_normal(x.shape)
        # central difference: error h^2 times third derivatives (order 1e2 here) plus 1e-16 / h
        assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-7
        if norm:
            u = r.standard_normal(8)
            assert abs((f(x, w + h * u) - f(x, w - h * u)) / (2 * h) - (dw * u).sum()) < 1e-7


def test_rotation_keeps_lengths_and_differences_of_positions():
    """|R x| = |x|, and (R_p x).(R_t y) depends on p - t alone."""
    r = np.random.default_rng(6)
    x, y = r.standard_normal((2, 16))
    fr = qk.frequencies(16, 10000.0)
    m = qk.matrices([5, 2, 105, 102], 16, 16, fr, False, 1.0)
    np.testing.assert_allclose(np.linalg.norm(m @ x, axis=1), np.linalg.norm(x), rtol=1e-12)
    np.testing.assert_allclose((m[0] @ x) @ (m[1] @ y), (m[2] @ x) @ (m[3] @ y), rtol=1e-12)
