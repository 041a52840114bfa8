"""Plain float64 RMS norm of heads with a position rotation, and its gradient.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

x [S, H, d], positions [S]: n = x r (w + w_offset) with r = 1 / sqrt(mean(x^2) +
eps) (or n = x), then element pairs (a, b) of the first rot elements become
(a c - b s, b c + a s), c + i s = rot_scale exp(i position inv_freq).  The
rotation is written as one matrix per position, so its gradient is the
transposed matrix.
"""
import math

import numpy as np


def pairs(rot, interleaved):
    if interleaved:
        return [(2 * i, 2 * i + 1) for i in range(rot // 2)]
    return [(i, i + rot // 2) for i in range(rot // 2)]


def frequencies(rot, base):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def matrices(positions, d, rot, inv_freq, interleaved, rot_scale):
    m = np.zeros((len(positions), d, d))
    m[:] = np.eye(d)
    for i, (a, b) in enumerate(pairs(rot, interleaved)):
        for t, pos in enumerate(positions):
            angle = int(pos) * inv_freq[i]     # to 2^-53 of itself
            c, s = rot_scale * math.cos(angle), rot_scale * math.sin(angle)
            m[t, a, a], m[t, a, b], m[t, b, a], m[t, b, b] = c, -s, s, c
    return m


def forward(x, w, m, eps, norm=True, w_offset=0.0):
    x = np.asarray(x, dtype=np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
        x = x * (1.0 if w is None else np.asarray(w, dtype=np.float64) + w_offset)
    return np.einsum("tab,thb->tha", m, x)


def backward(x, w, m, eps, dy, norm=True, w_offset=0.0):
    """(dx, dw)."""
    g = np.einsum("tba,thb->tha", m, np.asarray(dy, dtype=np.float64))
    if not norm:
        return g, None
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    xr = x * r
    h = g * (1.0 if w is None else np.asarray(w, dtype=np.float64) + w_offset)
    return r * (h - xr * (h * xr).mean(axis=-1, keepdims=True)), (g * xr).sum(axis=(0, 1))
