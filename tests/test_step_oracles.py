"""Pins of the oracles of linear attention, sampled acceptance and page planning, without a GPU:
each against statements that do not share its loop."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle.sample import UNIT, draw, units


def test_linear_is_the_sum_over_earlier_rows():
    rng = np.random.default_rng(1)
    n, H, Hk, dk, dv = 9, 4, 2, 5, 3
    q, k = rng.standard_normal((2, n, Hk, dk))
    v, g = rng.standard_normal((n, H, dv)), -rng.random((n, H))
    s0 = rng.standard_normal((2, H, dk, dv))
    cu = [0, 4, 9]
    o, s, mag, size = oracle.linear_attention(q, k, v, g, s0, cu, scale=0.5)
    for r in range(2):
        for h in range(H):
            for i in range(cu[r], cu[r + 1]):
                want = np.exp(g[cu[r]:i + 1, h].sum()) * (q[i, h // 2] @ s0[r, h])
                for j in range(cu[r], i + 1):
                    want = want + np.exp(g[j + 1:i + 1, h].sum()) * (q[i, h // 2] @ k[j, h // 2]) * v[j, h]
                np.testing.assert_allclose(o[i, h], 0.5 * want, rtol=1e-12, atol=1e-13)
    assert np.all(np.abs(o) <= mag * (1 + 1e-12)) and np.all(np.abs(s) <= size * (1 + 1e-12))


def test_linear_without_decay_of_some_rows():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 6, 1, 4))
    v, s0 = rng.standard_normal((6, 1, 4)), rng.standard_normal((2, 1, 4, 4))
    _, s, _, _ = oracle.linear_attention(q, k, v, np.zeros(1), s0, [0, 3, 6], rows=[0, 2])
    np.testing.assert_array_equal(s[0], s0[0])
    np.testing.assert_allclose(s[1, 0], s0[1, 0] + k[3:5, 0].T @ v[3:5, 0], rtol=1e-13)


def test_units_are_exact():
    for x in (0.0, 1.0, 0.5, 2.0 ** -44, 2.0 ** -45, 0.3, 1e-20, 0.999999):
        x = float(np.float32(x))
        assert units(x) == int(Fraction(x) * UNIT)
    assert units(float("nan")) == units(-1.0) == units(-0.0) == 0 and units(7.0) == UNIT


def test_draw_counts_every_weight():
    # each id is drawn by as many of the 2^31 random numbers as its share of the sum
    weights = [0, 3, 0, 1, 4, 0]
    ids = [draw(weights, (i + 0.5) / 8) for i in range(8)]
    assert ids == [1, 1, 1, 3, 4, 4, 4, 4]
    assert draw(weights, 1.0) == 4 and draw(weights, -1.0) == 1 and draw([0, 0], 0.5) == -1


@pytest.mark.parametrize("lookup", [False, True])
def test_accepted_tokens_follow_the_target(lookup):
    # what acceptance is for: whatever the drafts' distribution, the tokens follow p
    rng = np.random.default_rng(3)
    p = np.float32([0.1, 0.4, 0.05, 0.45])
    q = np.float32([0.4, 0.3, 0.2, 0.1])
    n = 20000
    drafts = np.full(n, 2) if lookup else rng.choice(4, n, p=q / q.sum(dtype=np.float64))
    ids = np.stack([np.zeros(n, int), drafts], 1).ravel()
    target, draft = np.tile(p, (2 * n, 1)), None if lookup else np.tile(q, (2 * n, 1))
    acc, nxt = oracle.accept_sample(ids, target, draft, rng.random(2 * n, np.float32),
                                    rng.random(n, np.float32), 2 * np.arange(n + 1))
    first = np.where(acc == 2, drafts, nxt)
    share = np.bincount(first, minlength=4) / n
    # four standard deviations of a share
    assert np.all(np.abs(share - p) <= 4 * np.sqrt(p * (1 - p) / n))
    assert set(acc) == {1, 2}


def test_pages_are_kept_apart():
    rng = np.random.default_rng(4)
    B, page, width, n_pages, max_T = 12, 16, 20, 120, 40
    free = list(rng.permutation(n_pages))
    kv_len, held, table = [0] * B, [0] * B, [[-1] * width for _ in range(B)]
    rows, accepted = [0] * B, [0] * B
    for step in range(30):
        accepted = [int(rng.integers(0, t + 1)) for t in rows]
        rows = [int(rng.integers(0, max_T + 1)) for _ in range(B)]
        over = (rng.random(B) < 0.1).astype(int)
        for r in range(B):  # room for what follows
            if kv_len[r] + accepted[r] + rows[r] > width * page:
                over[r] = 1
        p = oracle.plan_pages(kv_len, held, free, table, page, max_T, n_pages, rows, accepted, over)
        used = [x for r in range(B) for x in p["table"][r][:p["held"][r]]]
        assert sorted(used + p["free"]) == list(range(n_pages))
        assert len(set(p["slots"])) == len(p["slots"]) == p["cu"][-1]
        for r in range(B):
            T = p["cu"][r + 1] - p["cu"][r]
            assert p["kv_len"][r] == (0 if over[r] else kv_len[r] + accepted[r])
            assert p["kv_len"][r] + T <= p["held"][r] * page
            assert T in (0, rows[r])
            if T == 0 and not over[r] and rows[r] > 0:
                assert p["err"] & 256
        assert p["err"] in (0, 256)
        kv_len, held, free, table = p["kv_len"], p["held"], p["free"], p["table"]
        rows = [b - a for a, b in zip(p["cu"], p["cu"][1:])]
