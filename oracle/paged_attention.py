"""fp64 CPU oracle for the paged key-value cache, decode attention over it and
packed causal prompt attention — TEST INFRASTRUCTURE ONLY (see oracle/attention.py).

Definitions (per sequence, query head h, KV head j = h // (h_q / h_kv)):

* prompt attention of a queries over b keys: query i is at position i + b - a and
  attends over the keys 0 .. i + b - a; no such key: 0;
* a row of an 8-bit cache: the smallest power of two u >= 2^-126 for which the
  row's largest finite |x| is at most 448 u (u = 1 for a row without a non-zero
  finite value), and for each x the e4m3 number nearest to x / u, ties to the even
  code; NaN for an x that is not finite.  Found here by search in the table of all
  e4m3 numbers;
* position p of a sequence in the cache: slot p % page_size of page
  table[p // page_size].

Everything is widened exactly and evaluated in fp64; only visible entries are
ever read.
"""
import numpy as np

from .attention import _f64


def _lens(x):
    return [int(v) for v in (x.tolist() if hasattr(x, "tolist") else x)]


def e4m3_table():
    """The 256 values of the e4m3 format (no infinities; codes 0x7f and 0xff NaN)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** -9
        else:
            out[c] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


def quantise(x):
    """(values of the codes, exponents of the units) for rows x [..., D]."""
    x = _f64(x)
    finite = np.isfinite(x)
    amax = np.where(finite, np.abs(x), 0.0).max(axis=-1)
    # smallest e with amax <= 448 2^e: counted up through the exponents
    steps = np.arange(-126, 128)
    e = -126 + (amax[..., None] > 448.0 * 2.0 ** steps).sum(axis=-1)
    e = np.where(amax > 0, e, 0)
    y = np.where(finite, x, 0.0) / (2.0 ** e)[..., None]
    pos = e4m3_table()[:127]  # codes 0 .. 126: increasing
    hi = np.clip(np.searchsorted(pos, np.abs(y)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = pos[hi] - np.abs(y), np.abs(y) - pos[lo]
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    vals = np.copysign(pos[code], y)
    return np.where(finite, vals, np.nan), e


def dequantise(vals, e):
    return vals * (2.0 ** np.asarray(e, dtype=np.float64))[..., None]


def prompt(q, k, v, cu_q, cu_k, scale):
    """q [Tq, h_q, D]; k, v [Tk, h_kv, D]; offsets [N + 1].  Returns o [Tq, h_q, D] fp64."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    cq, ck = _lens(cu_q), _lens(cu_k)
    h_q, h_kv = q.shape[1], k.shape[1]
    o = np.zeros(q.shape)
    for n in range(len(cq) - 1):
        a, b = cq[n + 1] - cq[n], ck[n + 1] - ck[n]
        for h in range(h_q):
            j = h // (h_q // h_kv)
            for i0 in range(0, a, 256):
                i1 = min(a, i0 + 256)
                seen = np.clip(np.arange(i0, i1) + b - a + 1, 0, b)
                top = int(seen.max())
                if top == 0:
                    continue
                kk, vv = k[ck[n]:ck[n] + top, j], v[ck[n]:ck[n] + top, j]
                hidden = np.arange(top)[None] >= seen[:, None]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (q[cq[n] + i0:cq[n] + i1, h] @ np.where(np.isfinite(kk), kk, 0.0).T)
                    bad = ~np.isfinite(kk).all(axis=1)
                    if bad.any():  # a visible key that is not finite: its own products, no others'
                        s[:, bad] = scale * (q[cq[n] + i0:cq[n] + i1, h] @ kk[bad].T)
                    s = np.where(hidden, -np.inf, s)
                    m = s.max(axis=1, keepdims=True)
                    w = np.where(hidden, 0.0, np.exp(s - np.where(m == -np.inf, 0.0, m)))
                    tot = w.sum(axis=1, keepdims=True)
                    w = w / np.where(tot == 0, 1.0, tot)
                    r = w @ np.where(np.isfinite(vv), vv, 0.0)
                    for i in np.nonzero(~np.isfinite(vv).all(axis=1))[0]:  # added where visible
                        see = ~hidden[:, i]
                        r[see] += np.where(np.isfinite(vv[i]), 0.0, w[see, i][:, None] * vv[i][None])
                o[cq[n] + i0:cq[n] + i1, h] = r
    return o


def cached_rows(pages, table, length, page_size):
    """Rows 0 .. length - 1 of one sequence: pages [P, h_kv, page_size, D] (values) and the
    sequence's table -> [h_kv, length, D] fp64."""
    pages = np.asarray(pages, dtype=np.float64)
    t = _lens(table)
    out = np.zeros((pages.shape[1], length, pages.shape[3]))
    for p in range(length):
        out[:, p] = pages[t[p // page_size], :, p % page_size]
    return out


def decode(q, k_rows, v_rows, scale):
    """q [h_q, D] over k_rows, v_rows [h_kv, L, D]: o [h_q, D] fp64 (0 when L = 0)."""
    q = _f64(q)
    h_q, h_kv, L = q.shape[0], k_rows.shape[0], k_rows.shape[1]
    o = np.zeros(q.shape)
    for h in range(h_q):
        j = h // (h_q // h_kv)
        if L:
            s = scale * (k_rows[j] @ q[h])
            w = np.exp(s - s.max())
            o[h] = (w / w.sum()) @ v_rows[j]
    return o
