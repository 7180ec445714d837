"""Reading the error word of an attention layer's step through the C ABI."""
import ctypes

import pytest
import torch

from speculative_decode_gated_gb300 import binding
from test_attn_abi import fake, lib  # noqa: F401


def test_without_a_word(lib):  # noqa: F811
    code = ctypes.c_int32(9)
    assert lib.gdn_read_attn_error(ctypes.byref(fake(dev_err=None)), None, ctypes.byref(code)) == 0
    assert code.value == 0
    assert lib.gdn_read_attn_error(None, None, ctypes.byref(code)) == 1
    assert lib.gdn_read_attn_error(ctypes.byref(fake()), None, None) == 1


@pytest.mark.gpu
def test_errors_of_both_calls_are_read():
    from attn_cases import Case, to_dev
    c = Case(new=[2, 3], old=[20, 30], q_heads=4, kv_heads=2, hd=64, seed=1).device().run()
    assert binding.gdn_read_attn_error(c.attn) == 0
    c.dlen[1] = -1
    c.run()
    assert binding.gdn_read_attn_error(c.attn) == binding.GDN_DEVERR_KV_LEN
    q, o = to_dev(c.q, c.dtype), torch.empty_like(c.o)
    kv = q[:, :2].contiguous()
    c.dtable[0, 1] = -3
    turn = binding.make_rope(inv_freq=torch.ones(32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.gdn_rope_append(c.attn, turn, q, kv, kv, o, stream=side)
    assert binding.gdn_read_attn_error(c.attn, stream=side) == \
        binding.GDN_DEVERR_KV_LEN | binding.GDN_DEVERR_PAGE
    status = binding.lib().gdn_read_attn_error(c.attn.ref, side.cuda_stream,
                                               ctypes.byref(ctypes.c_int32()))
    assert status == binding.GDN_ERR_DEVICE_ARG
    c.derr.zero_()
    assert binding.gdn_read_attn_error(c.attn) == 0
    d = Case(new=[1], old=[4], q_heads=2, kv_heads=1, hd=64).device(err=False).run()
    assert binding.gdn_read_attn_error(d.attn) == 0
