"""Acceptance of sampled drafts (CPU oracle), in Python's whole numbers and fractions.

TEST INFRASTRUCTURE, like the rest of this package: only `tests/` and
`__graft_entry__.smoke()` use it.

Parity unpinned: none.  Pinned by `tests/test_step_oracles.py`.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

UNIT = 1 << 44


def units(x: float) -> int:
    """Whole units of 2^-44; NaN and below 0: none, above 1: as 1."""
    x = float(x)
    if not x > 0.0:
        return 0
    return UNIT if x > 1.0 else int(Fraction(x) * UNIT)


def below(u: float, q: float, p: float) -> bool:
    """u q < p, exactly; with NaN, or 0 times infinity, it is not."""
    if all(np.isfinite([u, q, p])):
        return Fraction(u) * Fraction(q) < Fraction(p)
    return u * q < p


def draw(weights, u: float) -> int:
    """The lowest i with w_0 + ... + w_i > floor(U W / 2^31), U = floor(2^31 u); -1 without weight."""
    total = sum(weights)
    if total == 0:
        return -1
    u = float(u)
    big = int(Fraction(min(u, 1.0)) * (1 << 31)) if u > 0.0 else 0
    border = min(big, (1 << 31) - 1) * total >> 31
    run = 0
    for i, w in enumerate(weights):
        run += w
        if run > border:
            return i
    raise AssertionError("the border lies below the sum")


def accept_sample(draft_ids, target, draft, u_accept, u_sample, cu):
    """target, draft (or None): [N, vocab]; returns (accepted [B], next ids [B])."""
    vocab = np.shape(target)[1]
    accepted, following = [], []
    for r in range(len(cu) - 1):
        c, T = int(cu[r]), int(cu[r + 1] - cu[r])
        if T == 0:
            accepted.append(0)
            following.append(-1)
            continue
        a, x = 1, None
        while a < T:
            x = int(draft_ids[c + a])
            if not 0 <= x < vocab:
                break
            p, u = float(target[c + a - 1][x]), float(u_accept[c + a])
            q = 1.0 if draft is None else float(draft[c + a - 1][x])
            if not below(u, q, p):
                break
            a += 1
        row = c + a - 1
        full = [units(p) for p in target[row]]
        w = full
        if a < T:
            if draft is None:
                w = [0 if i == x else p for i, p in enumerate(full)]
            else:
                w = [max(p - units(q), 0) for p, q in zip(full, draft[row])]
            if not any(w):
                w = full
        accepted.append(a)
        following.append(draw(w, u_sample[r]))
    return np.array(accepted, np.int32), np.array(following, np.int32)
