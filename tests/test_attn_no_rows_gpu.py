"""GPU: a ragged step whose maximum of rows is 0, over rows that no request has (a buffer that
is larger than its contents): nothing is written, and a request with rows is flagged."""
import pytest
import torch

from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [0, 2])
@pytest.mark.parametrize("max_pages", [4, 1000])
def test_max_T_of_zero(dtype, rows, max_pages):
    pages = [torch.zeros((4, 1, 16, 64), dtype=dtype, device="cuda") for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    attn = binding.make_attn(
        q_heads=2, k_pages=pages[0], v_pages=pages[1],
        page_table=torch.zeros((2, max_pages), dtype=torch.int32, device="cuda"),
        kv_len=torch.tensor([3, 5], dtype=torch.int32, device="cuda"), max_T=0,
        cu_seqlens=torch.tensor([0, 0, rows], dtype=torch.int32, device="cuda"), n_tok=8, dev_err=err)
    q = torch.ones((8, 2, 64), dtype=dtype, device="cuda")
    o = torch.full_like(q, 7.0)
    lse = torch.full((8, 2), 7.0, device="cuda")
    binding.gdn_paged_attn(attn, q, o, lse=lse, workspace=binding.paged_attn_workspace(attn))
    torch.cuda.synchronize()
    assert torch.all(o == 7) and torch.all(lse == 7)
    assert int(err.item()) == (binding.GDN_DEVERR_SEQLEN if rows else 0)
