"""fp64 CPU oracle for the norms and the rotation of q's and k's heads — TEST
INFRASTRUCTURE ONLY (see oracle/attention.py).

    y = w x / sqrt(mean x^2 + eps)   (without eps: y = x)
    pairs (a, b) of the first 2 n values, i = 0 .. n - 1: (i, i + n), or (2 i, 2 i + 1);
    y_a' + j y_b' = (y_a + j y_b) exp(j p_i f_i)

The angle is reduced in exact rationals (a position times a 32-bit frequency, over 2 pi to
70 digits), so that far positions lose nothing.
"""
from fractions import Fraction

import numpy as np

from .attention import _f64


def _pi():
    def arctan_inverse(x, one):
        term, total, n, sign = one // x, 0, 1, 1
        while term:
            total += sign * (term // n)
            term //= x * x
            n, sign = n + 2, -sign
        return total

    one = 10 ** 80
    return Fraction(4 * (4 * arctan_inverse(5, one) - arctan_inverse(239, one)), one)


TWO_PI = 2 * _pi()


def angle(position, freq):
    """position * freq in radians, mod 2 pi, for an integer and a float."""
    turns = Fraction(int(position)) * Fraction(float(freq)) / TWO_PI
    return float((turns - round(turns)) * TWO_PI)


def normed(x, weight, eps):
    x = _f64(x)
    if eps is None:
        return x
    top = np.abs(x).max(axis=-1, keepdims=True)
    unit = np.where((top > 0) & np.isfinite(top), top, 1.0)
    r = np.sqrt(np.mean((x / unit) ** 2, axis=-1, keepdims=True) + eps / unit ** 2)
    y = x / unit / r
    return y if weight is None else y * _f64(weight)


def rotate(x, positions, inv_freq, axes=None, interleaved=False, weight=None, eps=None):
    """x [T, h, D]; positions [T], or [A, T] with axes (one for each frequency).  Returns (the
    rotated heads, |y_a| + |y_b| of the pair that each value belongs to: 0 outside) in fp64."""
    y = normed(x, weight, eps)
    f = [float(v) for v in inv_freq]
    n, p = len(f), np.atleast_2d(np.asarray(positions))
    theta = np.array([[angle(p[axes[i] if axes is not None else 0, t], f[i]) for i in range(n)]
                      for t in range(y.shape[0])]).reshape(y.shape[0], 1, n)
    a = np.arange(n) * (2 if interleaved else 1)
    b = a + (1 if interleaved else n)
    out, size = y.copy(), np.zeros_like(y)
    c, s = np.cos(theta), np.sin(theta)
    with np.errstate(invalid="ignore"):
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size
