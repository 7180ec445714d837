"""Pins of the attention oracle (no GPU): closed forms, invariances and properties that
its definition has to have, and the frequency scalings."""
import numpy as np
import pytest

import oracle
from speculative_decode_gated_gb300 import staging


def cache(rng, lens, kv_heads=2, hd=8, page=4):
    need = [-(-n // page) for n in lens]
    ids = rng.permutation(sum(need) + 2)
    table = np.zeros((len(lens), max(need) + 1), np.int32)
    at = 0
    for r, k in enumerate(need):
        table[r, :k] = ids[at:at + k]
        at += k
    shape = (len(ids), kv_heads, page, hd)
    return rng.standard_normal(shape), rng.standard_normal(shape), table


def test_one_place_returns_its_value():
    rng = np.random.default_rng(0)
    k, v, table = cache(rng, [1])
    q = rng.standard_normal((1, 4, 8))
    o, lse, mean = oracle.paged_attention(q, [0, 1], [0], k, v, table, 0.3)
    for h in range(4):
        np.testing.assert_allclose(o[0, h], v[table[0, 0], h // 2, 0], rtol=1e-14)
        np.testing.assert_allclose(lse[0, h], 0.3 * q[0, h] @ k[table[0, 0], h // 2, 0], rtol=1e-13)
        np.testing.assert_allclose(mean[0, h], np.abs(o[0, h]), rtol=1e-14)


def test_equal_scores_average_the_visible_values():
    rng = np.random.default_rng(1)
    k, v, table = cache(rng, [11])
    q = np.zeros((3, 2, 8))
    rows = oracle.cached_rows(v, table, 0, 11)
    o, lse, _ = oracle.paged_attention(q, [0, 3], [8], k, v, table, 1.0)
    for t in range(3):
        np.testing.assert_allclose(o[t], rows[:9 + t].mean(0), rtol=1e-12)
        np.testing.assert_allclose(lse[t], np.log(9 + t), rtol=1e-12)
    o, _, _ = oracle.paged_attention(q, [0, 3], [8], k, v, table, 1.0, window=3, sinks=2)
    for t in range(3):
        c = [j for j in range(9 + t) if j > 8 + t - 3 or j < 2]
        np.testing.assert_allclose(o[t], rows[c].mean(0), rtol=1e-12)


def test_chunk_equals_one_token_at_a_time_and_a_wide_window():
    rng = np.random.default_rng(2)
    k, v, table = cache(rng, [9, 6])
    q = rng.standard_normal((7, 4, 8))
    cu, old = [0, 4, 7], [5, 3]
    o, lse, _ = oracle.paged_attention(q, cu, old, k, v, table, 0.5)
    for r in range(2):
        for t in range(cu[r + 1] - cu[r]):
            one, l1, _ = oracle.paged_attention(q[cu[r] + t][None], [0, 1], [old[r] + t], k, v,
                                                table[r:r + 1], 0.5)
            np.testing.assert_allclose(one[0], o[cu[r] + t], rtol=1e-12)
            np.testing.assert_allclose(l1[0], lse[cu[r] + t], rtol=1e-12)
    w, _, _ = oracle.paged_attention(q, cu, old, k, v, table, 0.5, window=100)
    np.testing.assert_array_equal(w, o)


def test_unseen_places_are_not_read():
    rng = np.random.default_rng(3)
    k, v, table = cache(rng, [10])
    q = rng.standard_normal((1, 2, 8))
    a = oracle.paged_attention(q, [0, 1], [6], k, v, table, 0.5, window=2, sinks=1)[0]
    for c in (1, 2, 3, 4, 7, 8, 9):
        k[table[0, c // 4], :, c % 4] = np.nan
        v[table[0, c // 4], :, c % 4] = np.nan
    b = oracle.paged_attention(q, [0, 1], [6], k, v, table, 0.5, window=2, sinks=1)[0]
    np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_lengths_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(4)
    f = 10000.0 ** (-np.arange(4) / 4.0)
    x, y = rng.standard_normal((2, 1, 3, 12))
    at = lambda z, p: oracle.rope(z, [p], f, interleaved)  # noqa: E731
    np.testing.assert_array_equal(at(x, 0), x)
    np.testing.assert_array_equal(at(x, 5)[..., 8:], x[..., 8:])
    np.testing.assert_allclose((at(x, 77) ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
    d = [(at(x, p + 9) * at(y, p)).sum(-1) for p in (0, 1, 1000)]
    np.testing.assert_allclose(d[0], d[1], rtol=1e-9)
    np.testing.assert_allclose(d[0], d[2], rtol=1e-8)
    # a quarter turn of the first pair: (x, y) -> (-y, x)
    z = oracle.rope(x, [1], [np.pi / 2], interleaved, mscale=2.0)
    np.testing.assert_allclose(z[..., 0], -2 * x[..., 1], rtol=1e-12)
    np.testing.assert_allclose(z[..., 1], 2 * x[..., 0], rtol=1e-12)


def test_halves_and_neighbours_are_the_same_up_to_order():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 3, 8))
    f = [0.3, 0.1, 0.02, 0.5]
    order = [0, 4, 1, 5, 2, 6, 3, 7]  # halves -> neighbours
    a = oracle.rope(x, [3, 9], f)[..., order]
    np.testing.assert_allclose(a, oracle.rope(x[..., order], [3, 9], f, True), rtol=1e-13)


def test_write_then_read():
    rng = np.random.default_rng(6)
    k, _, table = cache(rng, [4, 10])
    rows = rng.standard_normal((5, 2, 8))
    before = oracle.cached_rows(k, table, 1, 10)
    oracle.write_rows(k, table, 1, 3, rows)
    after = oracle.cached_rows(k, table, 1, 10)
    np.testing.assert_array_equal(after[3:8], rows)
    np.testing.assert_array_equal(after[:3], before[:3])
    np.testing.assert_array_equal(after[8:], before[8:])


def test_frequency_scalings():
    plain, one = staging.rope_frequencies(64, 10000.0)
    assert one == 1.0 and plain[0] == 1.0
    np.testing.assert_allclose(plain.numpy(), 10000.0 ** (-np.arange(32) / 32.0), rtol=1e-6)
    lin, one = staging.rope_frequencies(64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin.numpy(), plain.numpy() / 4, rtol=1e-6)
    ntk, one = staging.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0
    np.testing.assert_allclose(ntk[-1].item(), plain[-1].item() / 4, rtol=1e-5)
    yarn, m = staging.rope_frequencies(64, scaling="yarn", factor=4.0, trained=4096)
    np.testing.assert_allclose(m, 0.1 * np.log(4.0) + 1)
    turns = 4096 * plain.numpy() / (2 * np.pi)
    np.testing.assert_allclose(yarn.numpy()[turns >= 32], plain.numpy()[turns >= 32], rtol=1e-6)
    np.testing.assert_allclose(yarn.numpy()[turns <= 1], plain.numpy()[turns <= 1] / 4, rtol=1e-6)
    assert np.all(yarn.numpy() <= plain.numpy()) and np.all(yarn.numpy() >= plain.numpy() / 4.0001)
    for bad in (dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            staging.rope_frequencies(**bad)
