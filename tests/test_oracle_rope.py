"""Pins of the oracle of norms and rotations: known angles, invariants, relative positions."""
import math

import numpy as np
import pytest

from oracle.rope import TWO_PI, angle, normed, rotate


def test_angles():
    assert float(TWO_PI) == 2 * math.pi
    assert angle(0, 0.3) == 0 and angle(1, 0.5) == 0.5 and angle(-3, 0.25) == -0.75
    assert abs(angle(7, 1.0) - (7 - 2 * math.pi)) < 1e-15
    # 2 pi is near 710 / 113; a far position by the addition theorem, 2^30 = (2^15)^2
    assert abs(angle(710, 1.0) - (710 - 113 * 2 * math.pi)) < 1e-12
    z = complex(math.cos(angle(2 ** 15, 1.0)), math.sin(angle(2 ** 15, 1.0)))
    w = z ** 32768
    far = angle(2 ** 30, 1.0)
    assert abs(w / abs(w) - complex(math.cos(far), math.sin(far))) < 1e-10


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 16))
    f = [1.0, 0.25, 1e-3]
    y, size = rotate(x, [5, -7, 0], f, interleaved=interleaved)
    assert np.array_equal(y[2], x[2]) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-14)  # lengths stay
    a, b = (0, 1) if interleaved else (0, 3)
    assert np.allclose(y[0, :, a], x[0, :, a] * math.cos(5) - x[0, :, b] * math.sin(5), atol=1e-14)
    assert np.allclose(y[0, :, b], x[0, :, b] * math.cos(5) + x[0, :, a] * math.sin(5), atol=1e-14)
    assert np.all(size[..., 6:] == 0) and np.allclose(size[..., a], np.abs(x[..., a]) + np.abs(x[..., b]))
    # dot products go by the difference of positions alone
    q, k = x[:1], x[1:2]
    dots = [(rotate(q, [p], f, interleaved=interleaved)[0] * rotate(k, [p - 9], f, interleaved=interleaved)[0]).sum()
            for p in (9, 1000, 123456789)]
    assert np.allclose(dots, dots[0], rtol=1e-12)


def test_axes():
    rng = np.random.default_rng(1)
    x, f = rng.standard_normal((2, 1, 8)), [0.5, 0.25, 0.125, 1.0]
    pos = np.array([[3, 4], [10, -2], [7, 7]])
    y, _ = rotate(x, pos, f, axes=[0, 2, 1, 1])
    for t in range(2):
        for i, ax in enumerate([0, 2, 1, 1]):
            z = complex(x[t, 0, i], x[t, 0, i + 4]) * np.exp(1j * pos[ax, t] * f[i])
            assert abs(z - complex(y[t, 0, i], y[t, 0, i + 4])) < 1e-14


def test_norm():
    x = np.array([[3.0, 4.0, 0.0, 0.0], [0.0] * 4, [1e30, 0, 0, 0], [1e-30, 0, 0, 0]])
    y = normed(x, [1, 2, 3, 4], 1e-6)
    assert np.allclose(y[0], np.array([3, 8, 0, 0]) / math.sqrt(25 / 4 + 1e-6)) and np.all(y[1] == 0)
    assert np.allclose(y[2, 0], 2) and np.allclose(y[3, 0], 1e-27)
    assert np.allclose(normed(x[3:], None, 0.0)[0, 0], 2)
