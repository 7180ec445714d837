"""GPU: infinite values at places that a row sees.  By the definition (every weight is
above zero) an infinite value makes its element of the row's output infinite, with its sign, and
infinities of both signs or a NaN make it NaN, wherever in a tile the place lies: in one
that every row sees, or in one that some rows see in part.  Where the weight is below float32's
range the element may be NaN, but never finite."""
import numpy as np
import pytest

from attn_cases import Case

pytestmark = pytest.mark.gpu

# One row a key head, a tile of 16, drafts and a prompt on the tensor cores, wide heads.
SHAPES = [("bf16", 64, 1, 1), ("bf16", 128, 4, 4), ("bf16", 32, 9, 2), ("bf16", 256, 16, 2),
          ("bf16", 64, 16, 4), ("bf16", 128, 16, 8), ("bf16", 128, 150, 2), ("bf16", 64, 150, 3),
          ("fp32", 64, 1, 1), ("fp32", 128, 20, 3)]
OLD = 300


def case(dtype, hd, T, G, window=0, **kw):
    return Case(new=[T], old=[OLD], q_heads=2 * G, kv_heads=2, hd=hd, dtype=dtype, window=window,
                sinks=2 if window else 0, page=32, seed=hd + T, **kw)


def put(c, place, element, value):
    """At one place of key head 1."""
    c.v[c.table[0, place // c.page], 1, place % c.page, element] = value


def places(T):
    """In a tile that every row sees; one that only the last row's tile may cut; a row's own."""
    return [3, 100, OLD - 1, OLD + T // 2, OLD + T - 1]


@pytest.mark.parametrize("dtype,hd,T,G", SHAPES)
@pytest.mark.parametrize("window", [0, 290])
def test_an_infinite_value_keeps_its_sign(dtype, hd, T, G, window):
    for i, place in enumerate(places(T)):
        c = case(dtype, hd, T, G, window)
        if np.isnan(c.v[c.table[0, place // 32], 1, place % 32, 0]):
            continue  # behind every row's window
        value = np.inf if i % 2 else -np.inf
        put(c, place, 3, value)
        put(c, place, hd - 2, -value)
        c.device().run()
        got = c.o.float().cpu().numpy()
        rows = OLD + np.arange(T)
        sees = (place <= rows) & ((window == 0) | (place > rows - window) | (place < c.sinks))
        assert sees.any()
        assert np.all(got[sees][:, G:, 3] == value), (place, got[sees][:, G:, 3])
        assert np.all(got[sees][:, G:, hd - 2] == -value), place
        others = np.delete(got, [3, hd - 2], -1)
        assert np.all(np.isfinite(others)) and np.all(np.isfinite(got[:, :G]))
        assert np.all(np.isfinite(got[~sees]))
        c.check(rows=~sees)


@pytest.mark.parametrize("dtype,hd,T,G", SHAPES)
def test_both_signs_make_nan(dtype, hd, T, G):
    c = case(dtype, hd, T, G)
    put(c, 40, 5, np.inf)
    put(c, 200, 5, -np.inf)
    c.device().run()
    got = c.o.float().cpu().numpy()
    assert np.all(np.isnan(got[:, G:, 5])) and np.all(np.isfinite(np.delete(got, 5, -1)))


@pytest.mark.parametrize("dtype,hd,T,G", SHAPES)
def test_a_weight_below_the_range_does_not_hide_it(dtype, hd, T, G):
    # scores of some hundred units: most weights are zero in float32
    for place in places(T):
        c = case(dtype, hd, T, G, qscale=200.0)
        put(c, place, 3, np.inf)
        c.device().run()
        got = c.o.float().cpu().numpy()
        sees = place <= OLD + np.arange(T)
        assert not np.any(np.isfinite(got[sees][:, G:, 3])), place
        assert np.all(np.isfinite(got[~sees])) and np.all(np.isfinite(np.delete(got, 3, -1)))
