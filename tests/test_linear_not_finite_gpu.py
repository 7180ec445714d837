"""Outputs of drafts (gdn_linear_verify, fewer than 48 rows) whose values or keys are not finite: rows
before such a row keep every bit, and from it on the column (a key: the head) is not finite, as by the
definition, whose states are not finite from that row on."""
import pytest
import torch

from speculative_decode_gated_gb300 import binding
from test_linear_gpu import Case

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def outputs(bad, T, dtype, dk, dv):
    c = Case(new=[T, T, T - 1], heads=2, dk=dk, dv=dv, seed=21, dtype=dtype)
    for row, head, column, x in bad:
        c.dv_[row, head, column] = x
    o = c.output()
    binding.gdn_linear_verify(c.lin, o)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    return c, o


@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 128, 128), ("bf16", 64, 192), ("bf16", 128, 96), ("fp32", 64, 64)])
@pytest.mark.parametrize("T,at", [(2, 1), (12, 6), (16, 15), (17, 16), (40, 0), (40, 20), (47, 46)])
def test_a_value_reaches_its_own_row_and_later_ones(T, at, dtype, dk, dv):
    bad = [(T + at, 0, 3, INF), (T + at, 1, dv - 1, NAN), (2 * T + min(at, T - 2), 1, 17, -INF)]
    c, o = outputs(bad, T, dtype, dk, dv)
    _, ref = outputs([], T, dtype, dk, dv)
    changed = torch.zeros_like(o, dtype=torch.bool)
    ends = {1: 2 * T, 2: 3 * T - 1}
    for row, head, column, x in bad:
        changed[row:ends[row // T], head, column] = True
    assert torch.equal(o[~changed], ref[~changed])
    assert not bool(torch.isfinite(o[changed]).any())


@pytest.mark.parametrize("T,at", [(12, 6), (40, 20)])
@pytest.mark.parametrize("x", [INF, NAN])
def test_a_key_reaches_its_own_row_and_later_ones(T, at, x):
    c = Case(new=[T, T], heads=2, seed=22)
    c.dk_[T + at, 1, 5] = x
    ref = Case(new=[T, T], heads=2, seed=22)
    o, o_ref = c.output(), ref.output()
    binding.gdn_linear_verify(c.lin, o)
    binding.gdn_linear_verify(ref.lin, o_ref)
    changed = torch.zeros_like(o, dtype=torch.bool)
    changed[T + at:2 * T, 1] = True
    assert torch.equal(o[~changed], o_ref[~changed])
    assert not bool(torch.isfinite(o[changed]).any())
