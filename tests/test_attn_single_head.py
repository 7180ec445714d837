"""Caches with a single key head whose pages came from another order of the axes: the page is
contiguous all the same, whatever stride the axis of one carries (no GPU)."""
import pytest
import torch

from speculative_decode_gated_gb300 import binding


def attn(k, v):
    return binding.make_attn(q_heads=4, k_pages=k, v_pages=v, page_table=torch.zeros(3, 2, dtype=torch.int32),
                             kv_len=torch.zeros(3, dtype=torch.int32), max_T=2)


def test_pages_of_rows_of_one_head():
    k, v = (torch.zeros(5, 16, 1, 64).transpose(1, 2) for _ in range(2))
    assert k.stride(1) == 64
    a = attn(k, v)
    assert (a.c.kv_heads, a.c.page_size, a.c.page_stride) == (1, 16, 16 * 64)
    both = torch.zeros(5, 2, 16, 1, 64)
    a = attn(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
    assert a.c.page_stride == 2 * 16 * 64


@pytest.mark.parametrize("bad", [torch.zeros(5, 16, 2, 64).transpose(1, 2),   # rows of two heads
                                 torch.zeros(5, 1, 16, 128)[..., :64],        # rows apart
                                 torch.zeros(5, 1, 64, 16).transpose(2, 3)])
def test_pages_that_are_not_contiguous(bad):
    with pytest.raises(ValueError, match="contiguous"):
        attn(bad, bad.clone(memory_format=torch.preserve_format))
