"""Linear attention with a decay for each head (CPU oracle), row by row in float64.

TEST INFRASTRUCTURE, like the rest of this package: only `tests/` and
`__graft_entry__.smoke()` use it.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t

Parity unpinned: none.  Pinned by `tests/test_step_oracles.py`.
"""
from __future__ import annotations

import numpy as np


def linear_attention(q, k, v, log_decay, s0, cu, scale=1.0, rows=None):
    """q, k [N, k_heads, dk], v [N, heads, dv], log_decay [heads] or [N, heads], s0 [B, heads, dk,
    dv], row offsets cu [B+1]; rows [B]: how many of each request's rows to run (all when None).

    Returns (o [N, heads, dv], states [B, heads, dk, dv]) and the same two with every term taken
    by its absolute value: what rounding errors are relative to.  Rows not run are 0."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, group = v.shape[1], v.shape[1] // k.shape[1]
    g = np.broadcast_to(np.asarray(log_decay, np.float64), (v.shape[0], H))
    out, mag = np.zeros(v.shape), np.zeros(v.shape)
    states = np.array(s0, np.float64)
    sizes = np.abs(states)
    for r in range(len(cu) - 1):
        n = cu[r + 1] - cu[r] if rows is None else rows[r]
        for i in range(cu[r], cu[r] + n):
            for h in range(H):
                lam = np.exp(g[i, h])
                kk, qq = k[i, h // group], q[i, h // group]
                states[r, h] = lam * states[r, h] + np.outer(kk, v[i, h])
                sizes[r, h] = lam * sizes[r, h] + np.outer(np.abs(kk), np.abs(v[i, h]))
                out[i, h] = scale * (qq @ states[r, h])
                mag[i, h] = abs(scale) * (np.abs(qq) @ sizes[r, h])
    return out, states, mag, sizes
