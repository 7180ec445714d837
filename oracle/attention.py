"""Rotary positions and attention over a paged key/value cache in float64 (CPU oracle).

TEST INFRASTRUCTURE, like the rest of this package.  Plain numpy from the
definitions:

    pair (x, y) of a head at position p:  x cos a - y sin a,  x sin a + y cos a,  a = p f_i
    o_t = sum_j w_j v_j,  w = softmax over the visible places j of scale q_t . k_j

Place c of request r lies in page table[r][c // P], row c % P of the pages
[n_pages][kv_heads][P][head_dim].

Parity unpinned: none.  Pinned by `tests/test_attn_oracle.py`.
"""
from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, interleaved=False, mscale=1.0) -> np.ndarray:
    """x: [N, heads, head_dim]; the first 2 len(inv_freq) elements of a head turn."""
    out = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)[None, :]
    c, s = (mscale * np.cos(a))[:, None, :], (mscale * np.sin(a))[:, None, :]
    u, w = out[..., first].copy(), out[..., second].copy()
    out[..., first] = u * c - w * s
    out[..., second] = u * s + w * c
    return out


def write_rows(pages, table, r, place0, rows) -> None:
    """Rows [T, kv_heads, head_dim] of request r to places place0, place0 + 1, ... (in place)."""
    P = pages.shape[2]
    for t in range(rows.shape[0]):
        c = place0 + t
        pages[table[r][c // P], :, c % P] = rows[t]


def cached_rows(pages, table, r, n) -> np.ndarray:
    """The first n places of request r: [n, kv_heads, head_dim]."""
    P = pages.shape[2]
    return np.stack([pages[table[r][c // P], :, c % P] for c in range(n)]) if n else \
        np.zeros((0, pages.shape[1], pages.shape[3]), pages.dtype)


def paged_attention(q, cu, kv_len, k_pages, v_pages, table, scale, window=0, sinks=0):
    """(o [N, q_heads, head_dim], lse [N, q_heads], mean_abs [N, q_heads, head_dim]):
    mean_abs is sum_j w_j |v_j|, the scale of a rounding of the weights."""
    q = np.asarray(q, np.float64)
    N, Hq, hd = q.shape
    G = Hq // k_pages.shape[1]
    o, lse, mean = np.zeros_like(q), np.zeros((N, Hq)), np.zeros_like(q)
    for r in range(len(cu) - 1):
        T, n0 = cu[r + 1] - cu[r], kv_len[r]
        if T <= 0:
            continue
        P = k_pages.shape[2]
        c = np.arange(n0 + T)
        needed = np.zeros(n0 + T, bool)  # places that some row sees: no other is read
        for t in range(T):
            needed |= _visible(c, n0 + t, window, sinks)
        at = c[needed]
        page = np.asarray(table[r])[at // P]
        k = np.asarray(k_pages[page, :, at % P], np.float64)  # [n, kv_heads, hd]
        v = np.asarray(v_pages[page, :, at % P], np.float64)
        for t in range(T):
            seen = _visible(at, n0 + t, window, sinks)
            for h in range(Hq):
                x = scale * (k[seen, h // G] @ q[cu[r] + t, h])
                m = x.max()
                with np.errstate(invalid="ignore"):  # a bad token makes the row NaN
                    e = np.exp(x - m)
                total = e.sum()
                o[cu[r] + t, h] = (e / total) @ v[seen, h // G]
                mean[cu[r] + t, h] = (e / total) @ np.abs(v[seen, h // G])
                lse[cu[r] + t, h] = m + np.log(total)
    return o, lse, mean


def _visible(j, p, window, sinks):
    """Which of the places j the row at place p sees."""
    seen = j <= p
    if window:
        seen &= (j > p - window) | (j < sinks)
    return seen
