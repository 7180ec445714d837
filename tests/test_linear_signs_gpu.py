"""Linear attention whose decays' logarithms have both signs: each decay between two rows is the
exponential of their sum, also where single decays, or those of some rows, are outside float32.

The logarithms are multiples of 1/4, so that all their sums are exact in float32, and a decay that float32
has is off by the exponential's 2^-22 alone: the tolerances of test_linear_gpu.py hold as they are.  A decay
below 2^-126 is off by up to 2^-149, the least float32 (e^-112 = 2^-161.6 is 0): that times the largest size
that a state of the case takes on, and for an output dk of these times the largest query, is allowed too."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gb300 import binding
from test_linear_drafts_gpu import Drafts
from test_linear_gpu import TILES

pytestmark = pytest.mark.gpu


class Signs(Drafts):
    """Two requests and heads with the logarithms given, [rows].  only: rows whose values are not 0 (None:
    all)."""

    def __init__(self, logs, only=None, **kw):
        super().__init__(new=[len(logs), len(logs)], heads=2, **kw)
        logs = np.tile(np.asarray(logs, np.float32), 2)
        self.g = np.ascontiguousarray(np.stack([logs, logs], 1))
        self.dg[:self.n] = torch.from_numpy(self.g).cuda()
        if only is not None:
            hidden = np.ones(len(logs), bool)
            hidden.reshape(2, -1)[:, list(only)] = False
            self.v[hidden] = 0.0
            self.dv_[:self.n][torch.from_numpy(hidden).cuda()] = 0.0
        self.largest = 0.0
        add = float(np.abs(self.k).max()) * np.abs(self.v).max((1, 2))
        for i, log in enumerate(logs):
            if i % (len(logs) // 2) == 0:  # a request's first row
                size = float(np.abs(self.s0).max())
            self.largest = max(self.largest, size)
            size = np.exp(float(log)) * size + float(add[i])
            self.largest = max(self.largest, size)

    def tolerance(self, value, mag, state):
        tiny = 2.0 ** -149 * self.largest
        if not state:
            tiny *= abs(self.scale) * self.dk * float(np.abs(self.q).max())
        return super().tolerance(value, mag, state) + tiny


def sums(*each):
    """32 rows for each sum, all alike (a sum is a multiple of 8)."""
    return np.repeat(np.asarray(each, np.float64) / 32, 32)


PROFILES = {
    # sums of 32 rows of which one is below and the others well within float32
    "deep_first": sums(-112, 24, 24, 24),
    "deep_last": sums(24, 24, 24, -112),
    "deep_between": sums(40, -112, 40, 24),
    # 32 rows that are not steep for themselves, but earlier ones of which are far above them
    "far_above": sums(40, 40, -56, -56),
    "far_above_then_flat": sums(56, 24, -40, 0),
    # two blocks of 128 rows, and an end within 32; without values only: a row's in the first 32
    # would be multiplied by up to e^(24 + 24 + 24 + 32) = 1e45, more than float32 has
    "long": np.concatenate([sums(-112, 24, 24, 24, 32, -112, 40, 24), sums(-24)[:17]]),
    "long_with_values": np.concatenate([sums(-112, 24, 24, 24, -112, 40, 24, -40), sums(-24)[:17]]),
    # far below, with small rises
    "small_rises": np.tile([-2, -2, 0.25, -4, -2, -6, 0.25, -2], 25),
    # a state that is forgotten in between
    "forgets": np.where(np.arange(160) == 50, -np.inf, np.concatenate([sums(40, -8, 24, 24), sums(-16)])),
    # up and down within 32 rows, further than 60 from their start
    "steep_up_and_down": np.tile(np.concatenate([np.full(16, 4.5), np.full(16, -4.5)]), 4),
}


@pytest.mark.parametrize("name,only", [(n, o) for n in sorted(PROFILES) for o in ("none", "first", "all")
                                       if n != "long" or o == "none"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_prompts(name, only, dk, dv):
    logs = PROFILES[name]
    assert len(logs) >= TILES and np.all(logs * 4 == np.round(logs * 4))
    rows = {"none": [], "first": range(32), "all": None}[only]
    c = Signs(logs, rows, dk=dk, dv=dv, seed=31)
    o = c.output()
    binding.gdn_linear_verify(c.lin, o)
    c.check(o)
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


@pytest.mark.parametrize("kept", [32, 64, 100, 128])
def test_a_prompt_s_commit(kept):
    c = Signs(PROFILES["deep_first"], [], seed=32)
    binding.gdn_linear_commit(c.lin, torch.tensor([kept, kept], dtype=torch.int32, device="cuda"))
    c.check(rows=[kept, kept])


@pytest.mark.parametrize("seed,reach", [(0, 28), (1, 28), (2, 8), (3, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [9, 16, 40, 300])
def test_walks(T, dtype, seed, reach):
    # a walk that stays within 2 reach of where it was at any earlier row
    rng = np.random.default_rng(40 + seed)
    logs, at = [], 0.0
    for _ in range(T):
        step = float(rng.integers(-8, 9)) / 4
        step = -abs(step) if at + step > reach else abs(step) if at + step < -reach else step
        logs.append(step)
        at += step
    c = Signs(logs, seed=seed, dtype=dtype, dk=64, dv=64)
    o = c.output()
    binding.gdn_linear_verify(c.lin, o)
    c.check(o)
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)
