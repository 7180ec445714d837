"""Strides whose arrays would span more than any address (no GPU): refused, so that the
checks for overlap never work with sums that have wrapped around."""
import pytest

from test_attn_abi import Q, attn, fake, lib, rope  # noqa: F401


@pytest.mark.parametrize("n_pages,page_stride", [(1 << 30, 1 << 33), ((1 << 31) - 1, 1 << 36), (1 << 28, 1 << 29)])
def test_pages(lib, n_pages, page_stride):  # noqa: F811
    c = fake(n_pages=n_pages, page_stride=page_stride)
    # the output lies within the span of the pages
    assert attn(lib, c, o=c.k_pages + page_stride) == 2
    assert rope(lib, c, o=c.k_pages + page_stride) == 2


@pytest.mark.parametrize("stride", [1 << 30, 1 << 36])
def test_rows(lib, stride):  # noqa: F811
    c = fake(batch=1 << 20, max_T=1 << 10, q_heads=2)
    assert attn(lib, c, q_stride=stride, o=Q + (1 << 20)) == 2
    assert rope(lib, c, sq=stride) == 2
    assert rope(lib, c, sq=256, sk=stride) == 2
    assert rope(lib, c, sq=256, sv=stride) == 2


def test_the_widest_that_fit(lib):  # noqa: F811
    # as far as the check for overlap: the output lies within them
    c = fake(n_pages=1 << 20, page_stride=1 << 36)
    assert attn(lib, c, o=c.k_pages + (1 << 36)) == 8
    c = fake()
    assert attn(lib, c, q_stride=1 << 36, o=Q + (1 << 36)) == 8
