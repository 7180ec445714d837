"""The blended (yarn) frequencies, pair by pair, against values worked out by hand.

With n elements, base b and L trained positions, pair i makes L b^(-2i / n) / (2 pi) turns,
so s turns belong to the index n ln(L / (2 pi s)) / (2 ln b).  From the index of 32 turns
rounded down to that of one turn rounded up, a pair's factor falls linearly from 1 to 1 / factor."""
import math

import numpy as np
import pytest

from speculative_decode_gated_gb300 import staging

CASES = [
    # n, base, L, factor, and by hand: 64 ln(20.372) / 9.2103 = 20.9, 64 ln(651.90) / 9.2103 = 45.03
    (128, 10000.0, 4096, 32.0, 20, 46),
    # 32 ln(162.97) / 13.8155 = 11.8, 32 ln(5215.2) / 13.8155 = 19.8
    (64, 1000000.0, 32768, 4.0, 11, 20),
    # 32 ln(20.372) / 9.2103 = 10.5, 32 ln(651.90) / 9.2103 = 22.5
    (64, 10000.0, 4096, 8.0, 10, 23),
    # below the first pair and 16 ln(15.915) / 13.1224 = 3.4
    (32, 500000.0, 100, 8.0, 0, 4),
]


@pytest.mark.parametrize("n,base,trained,factor,first,last", CASES)
def test_every_pair_of_the_ramp(n, base, trained, factor, first, last):
    f, mscale = staging.rope_frequencies(n, base, "yarn", factor, trained)
    want = []
    for i in range(n // 2):
        part = min(max((i - first) / (last - first), 0.0), 1.0)  # of the way to 1 / factor
        want.append(base ** (-2.0 * i / n) * (1.0 - part + part / factor))
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-6)
    assert abs(mscale - (0.1 * math.log(factor) + 1.0)) < 1e-12


def test_single_pairs():
    f, _ = staging.rope_frequencies(128, 10000.0, "yarn", 32.0, 4096)
    # pair 33 is half way from 20 to 46, pair 40 20 of 26 steps
    np.testing.assert_allclose(f[33].item(), 10000.0 ** (-66 / 128) * (1 + 1 / 32) / 2, rtol=1e-6)
    np.testing.assert_allclose(f[40].item(), 10000.0 ** (-80 / 128) * (6 + 20 / 32) / 26, rtol=1e-6)
    f, _ = staging.rope_frequencies(64, 1000000.0, "yarn", 4.0, 32768)
    np.testing.assert_allclose(f[14].item(), 1000000.0 ** (-28 / 64) * (6 + 3 / 4) / 9, rtol=1e-6)


def test_given_turns():
    # 16 ln(2048 / (2 pi 4)) / ln(10000) = 7.6, 16 ln(2048 / pi) / ln(10000) = 11.3
    f, _ = staging.rope_frequencies(32, 10000.0, "yarn", 2.0, 2048, beta_fast=4.0, beta_slow=0.5)
    part = np.clip((np.arange(16) - 7) / 5.0, 0, 1)
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(16) / 16.0) * (1 - part / 2), rtol=1e-6)


def test_blend_in_turns():
    f, _ = staging.rope_frequencies(128, 10000.0, "yarn_turns", 32.0, 4096)
    plain = 10000.0 ** (-np.arange(64) / 64.0)
    part = np.clip((4096 * plain / (2 * np.pi) - 1) / 31, 0, 1)
    np.testing.assert_allclose(f.numpy(), plain * (part + (1 - part) / 32), rtol=1e-6)


@pytest.mark.parametrize("over", [dict(beta_fast=1.0), dict(beta_slow=0.0), dict(beta_slow=40.0),
                                  dict(trained=6)])
@pytest.mark.parametrize("scaling", ["yarn", "yarn_turns"])
def test_refusals(over, scaling):
    with pytest.raises(ValueError):
        staging.rope_frequencies(64, scaling=scaling, factor=4.0, **over)
