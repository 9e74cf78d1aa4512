"""Pins of the oracle of attention over cached rows with a window: a loop over single keys,
the other oracles where they say the same, and values that nobody sees."""
import math

import numpy as np
import pytest

from oracle.paged_attention import decode, prompt
from oracle.window_attention import attend, seen


def brute(q, k, v, scale, window, sinks, gone):
    a, h_q, D = q.shape
    h_kv, L = k.shape[:2]
    o = np.zeros(q.shape)
    for i in range(a):
        p = L - a + i
        for h in range(h_q):
            j = h // (h_q // h_kv)
            keys = [x for x in range(max(0, p + 1)) if not gone[x] and
                    (not window or x > p - window or x < sinks)]
            w = [math.exp(scale * float(q[i, h] @ k[j, x])) for x in keys]
            for x, y in zip(keys, w):
                o[i, h] += y / sum(w) * v[j, x]
    return o


@pytest.mark.parametrize("a,L,window,sinks", [(1, 1, 0, 0), (3, 9, 0, 0), (4, 12, 3, 0), (4, 12, 3, 2), (12, 12, 1, 0),
                                              (5, 20, 6, 30), (7, 4, 2, 1), (2, 0, 0, 0)])
def test_brute_force(a, L, window, sinks):
    rng = np.random.default_rng(a * 100 + L)
    q, k, v = rng.standard_normal((a, 4, 6)), rng.standard_normal((2, L, 6)), rng.standard_normal((2, L, 6))
    gone = rng.random(L) < 0.2
    for g in (np.zeros(L, dtype=bool), gone):
        o, size = attend(q, k, v, 0.4, window, sinks, g)
        assert np.allclose(o, brute(q, k, v, 0.4, window, sinks, g), atol=1e-13)
        assert (size >= np.abs(o) - 1e-13).all()


def test_like_the_other_oracles():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((6, 4, 8)), rng.standard_normal((2, 10, 8)), rng.standard_normal((2, 10, 8))
    o = attend(q, k, v, 0.3)[0]
    assert np.allclose(o, prompt(q, k.transpose(1, 0, 2), v.transpose(1, 0, 2), [0, 6], [0, 10], 0.3), atol=1e-13)
    assert np.allclose(o[-1], decode(q[-1], k, v, 0.3), atol=1e-13)
    assert np.allclose(attend(q, k, v, 0.3, window=10, sinks=0)[0], o, atol=1e-13)
    assert np.allclose(attend(q, k, v, 0.3, window=1, sinks=0)[0], np.repeat(v[:, 4:].transpose(1, 0, 2), 2, axis=1))


def test_what_is_not_seen_has_no_effect():
    rng = np.random.default_rng(6)
    q, k, v = rng.standard_normal((2, 2, 4)), rng.standard_normal((1, 9, 4)), rng.standard_normal((1, 9, 4))
    want = attend(q, k, v, 1.0, 3, 1)[0]
    unseen = ~seen(2, 9, 3, 1).any(axis=0)
    assert unseen.tolist() == [False] + [True] * 4 + [False] * 4
    k[:, unseen], v[:, unseen] = np.nan, np.inf
    assert np.array_equal(attend(q, k, v, 1.0, 3, 1)[0], want)
    v[0, 5, 2] = np.inf  # the first query's window begins here, the second's behind
    got = attend(q, k, v, 1.0, 3, 1)[0]
    assert np.isinf(got[0, :, 2]).all() and np.array_equal(got[1], want[1])
