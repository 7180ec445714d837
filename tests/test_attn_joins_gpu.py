"""GPU parity of attention where a unit's places lie in many workers: joined by a launch of
its own (few units) or by the warpgroup that ends last (many), on every kernel; and one
workspace that all of them use in turn."""
import pytest
import torch

from attn_cases import Case
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


def few(hd, rows, kv_heads=1, dtype="bf16", **kw):
    return Case(new=[rows // 8], old=[21003], q_heads=8 * kv_heads, kv_heads=kv_heads, hd=hd, page=64,
                dtype=dtype, seed=rows + hd, **kw)


def many(hd, T, B=40, **kw):
    """One long request among short ones: its units span most of the workers."""
    old = [17 * r % 90 for r in range(B)]
    old[B // 3] = 15001
    return Case(new=[T if r % 5 else T // 2 for r in range(B)], old=old, q_heads=16, kv_heads=2,
                hd=hd, page=32, seed=T + hd, **kw)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [8, 40, 128, 136, 512])
@pytest.mark.parametrize("kv_heads", [1, 3])
def test_few_units(hd, rows, kv_heads):
    few(hd, rows, kv_heads).device().run().check()


@pytest.mark.parametrize("hd", [32, 256])
def test_few_units_other_heads(hd):
    few(hd, 16).device().run().check()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T", [1, 9, 16, 24])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9000, 5)])
def test_many_units(hd, T, window, sinks):
    many(hd, T, window=window, sinks=sinks).device().run().check()


def test_one_workspace_for_every_kernel():
    cases = [many(128, 16), few(128, 512), few(64, 128, dtype="bf16"), many(64, 24), few(128, 8),
             few(64, 16, dtype="fp32"), many(64, 1)]
    for c in cases:
        c.device()
    size = max(binding.paged_attn_workspace(c.attn).numel() for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for c in cases + cases[::-1]:
        c.run(workspace=ws).check()
