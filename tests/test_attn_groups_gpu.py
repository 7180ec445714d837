"""GPU parity of attention for groups of query heads that the tensor-core kernels cannot
fetch as boxes (a count that is not a power of two, or above 128), so that the softmax
warpgroups copy the queries themselves: drafts and prompt chunks, tokens that straddle the 128 rows
of a warpgroup, and workers that hold many units one after the other.  And the accuracy of the
16-row kernel, whose weights enter the second product in two terms."""
import numpy as np
import pytest

from attn_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G", [3, 5, 7, 12])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_prompt_chunks(hd, G, window, sinks):
    Case(new=[300, 0, 1, 171], old=[0, 40, 333, 77], q_heads=2 * G, kv_heads=2, hd=hd, page=32,
         window=window, sinks=sinks, seed=G + hd).device().run().check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G,T", [(3, 11), (5, 25), (7, 18), (20, 6)])
def test_drafts(hd, G, T):
    Case(new=[T, 1, T // 2, T], old=[0, 500, 129, 64], q_heads=3 * G, kv_heads=3, hd=hd,
         seed=G + T).device().run().check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G,T,B", [(3, 40, 400), (5, 25, 500), (3, 60, 150), (6, 130, 40)])
def test_many_units_a_worker(hd, G, T, B):
    rng = np.random.default_rng(G + T)
    new, old = rng.integers(0, T + 1, B), rng.integers(0, 60, B)
    new[3] = T
    Case(new=new.tolist(), old=old.tolist(), q_heads=2 * G, kv_heads=2, hd=hd,
         seed=T).device().run().check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("G,T", [(130, 1), (130, 2), (192, 3), (256, 2)])
def test_groups_above_a_warpgroup(hd, G, T):
    Case(new=[T, 1], old=[70, 9], q_heads=G, kv_heads=1, hd=hd, seed=G + T).device().run().check()


@pytest.mark.parametrize("hd,T,G", [(32, 1, 1), (32, 40, 2), (64, 1, 16), (64, 4, 3), (128, 1, 8),
                                    (128, 16, 1), (256, 1, 8), (256, 30, 2)])
@pytest.mark.parametrize("old", [60, 1500])
def test_weights_of_the_16_row_kernel_are_not_rounded_to_bf16(hd, T, G, old):
    # Only the output's rounding and the scores' error are left of attn_cases.check_close: the
    # weights' two terms leave 2^-16 of them.
    c = Case(new=[T, 1], old=[old, 33], q_heads=2 * G, kv_heads=2, hd=hd, seed=hd + T + old)
    c.device().run()
    o, _, mean = c.expected()
    got = c.o.float().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -11 * mean
    assert np.all(np.abs(got - o) <= tol), float(np.max(np.abs(got - o) / tol))
