"""fp64 CPU oracle for attention of new tokens over cached rows, all of them or a window and
the first few — TEST INFRASTRUCTURE ONLY (see oracle/attention.py).

The a queries of a sequence are the last a of its L positions; the query at position p sees
the keys j <= p, with window > 0 those of them with j > p - window or j < sinks, and never
a key whose page is gone.  o = sum_j softmax(scale q.k)_j v_j, 0 where nothing is seen.
"""
import numpy as np

from .attention import _f64


def seen(a, L, window, sinks, gone=None):
    """[a, L] truth values."""
    p, j = np.arange(L - a, L)[:, None], np.arange(L)[None]
    s = j <= p
    if window:
        s &= (j > p - window) | (j < sinks)
    return s if gone is None else s & ~np.asarray(gone, dtype=bool)[None]


def attend(q, k, v, scale, window=0, sinks=0, gone=None):
    """q [a, h_q, D]; k, v [h_kv, L, D].  Returns (o, the same sums over |v|) [a, h_q, D]."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    a, h_q, L = q.shape[0], q.shape[1], k.shape[1]
    see = seen(a, L, window, sinks, gone)
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    keys = np.nonzero(see.any(axis=0))[0]  # what nobody sees is not even read
    if len(keys) == 0:
        return o, size
    see = see[:, keys]
    for h in range(h_q):
        kk, vv = k[h // (h_q // k.shape[0])][keys], v[h // (h_q // k.shape[0])][keys]
        with np.errstate(invalid="ignore", over="ignore"):
            bad = ~np.isfinite(kk).all(axis=1)
            s = scale * (q[:, h] @ np.where(bad[:, None], 0.0, kk).T)
            for i in np.nonzero(bad)[0]:
                s[:, i] = scale * (q[:, h] @ kk[i])
            s = np.where(see, s, -np.inf)
            m = s.max(axis=1, keepdims=True)
            w = np.where(see, np.exp(s - np.where(m == -np.inf, 0.0, m)), 0.0)
            tot = w.sum(axis=1, keepdims=True)
            w = w / np.where(tot == 0, 1.0, tot)
            fine = np.where(np.isfinite(vv), vv, 0.0)
            r = w @ fine
            for i in np.nonzero(~np.isfinite(vv).all(axis=1))[0]:
                r[see[:, i]] += np.where(np.isfinite(vv[i]), 0.0, w[see[:, i], i][:, None] * vv[i][None])
            o[:, h], size[:, h] = r, w @ np.abs(fine)
    return o, size
