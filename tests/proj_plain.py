"""Projections with 4-bit weights and the rotation of heads in NumPy: fp64, from the definitions alone."""
from decimal import Decimal
from fractions import Fraction

import numpy as np

PI = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803"))


def int4_values(w, s):
    """uint8 [n, k / 2] nibbles and fp16 [n, k / 128] scales: the weights [n, k]."""
    w = np.asarray(w).astype(np.int64)
    q = np.empty((w.shape[0], w.shape[1] * 2))
    q[:, 0::2], q[:, 1::2] = w % 16, w // 16
    q[q >= 8] -= 16
    return q * np.repeat(np.asarray(s, np.float64), 128, axis=1)


def angles(freq, pos):
    """pos * freq mod a turn, in radians [-pi, pi]: exact until the last step."""
    out = np.empty((len(pos), len(freq)))
    for j, f in enumerate(freq):
        step = Fraction(float(f)) / (2 * PI)
        for i, p in enumerate(pos):
            t = int(p) * step
            t -= round(t)
            out[i, j] = float(2 * PI * t)
    return out


def rotate(x, freq, pos, *, interleaved=False, amp=1.0, norm=False, weight=None, eps=1e-6):
    """(y, size): x [tokens, heads, dim] rotated, and the size that its errors are relative to: |x_a| + |x_b| of a pair,
    after norm and amp."""
    x = np.asarray(x, np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * np.asarray(weight, np.float64)
    y, size = x.copy(), np.abs(x)
    n = len(freq)
    if n == 0:
        return y, size
    a = np.arange(n) * 2 if interleaved else np.arange(n)
    b = a + (1 if interleaved else n)
    t = angles(freq, pos)[:, None]
    y[..., a] = amp * (x[..., a] * np.cos(t) - x[..., b] * np.sin(t))
    y[..., b] = amp * (x[..., b] * np.cos(t) + x[..., a] * np.sin(t))
    both = abs(amp) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    size[..., a], size[..., b] = both, both
    return y, size
