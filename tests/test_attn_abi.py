"""The attention calls without a GPU: struct layouts, what the host validation refuses
before any CUDA call, and what the binding's own checks refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decode_gated_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, STEP = 1 << 44, 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import speculative_decode_gated_gb300 as pkg
        pkg.build()
    return binding.lib()


@pytest.mark.parametrize("cls", [binding.gdn_attn, binding.gdn_rope])
def test_struct_layout_matches_c(tmp_path, cls):
    name = cls.__name__
    fields = [f[0] for f in cls._fields_]
    prog = tmp_path / "layout.c"
    body = "\n".join(f'printf("%zu ", offsetof({name}, {f}));' for f in fields)
    prog.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "gdn.h"\n'
                    f'int main(void) {{ {body} printf("%zu\\n", sizeof({name})); return 0; }}\n')
    exe = tmp_path / "layout"
    cuda_inc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-I", cuda_inc, str(prog),
                    "-o", str(exe)], check=True)
    c_vals = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True,
                                             check=True).stdout.split()]
    assert c_vals == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


def fake(**over):
    """A step with plausible, aligned fake device addresses (never dereferenced)."""
    c = binding.gdn_attn()
    c.batch, c.q_heads, c.kv_heads, c.head_dim = 2, 8, 2, 128
    c.max_T, c.dtype, c.page_size, c.max_pages = 4, binding.GDN_BF16, 16, 10
    c.scale = 0.1
    c.n_tok = 8
    c.k_pages, c.v_pages, c.n_pages = BASE, BASE + STEP, 30
    c.page_stride = 2 * 16 * 128
    c.page_table, c.kv_len, c.dev_err = BASE + 2 * STEP, BASE + 3 * STEP, BASE + 4 * STEP
    for k, v in over.items():
        setattr(c, k, v)
    return c


def fake_rope(**over):
    r = binding.gdn_rope()
    r.rot_dim, r.interleaved, r.mscale = 128, 0, 1.0
    r.inv_freq = BASE + 5 * STEP
    for k, v in over.items():
        setattr(r, k, v)
    return r


Q, O, WS = BASE + 6 * STEP, BASE + 7 * STEP, BASE + 8 * STEP
K, V, LSE = BASE + 9 * STEP, BASE + 10 * STEP, BASE + 11 * STEP
CU = BASE + 12 * STEP


def attn(lib, c, q=Q, q_stride=1024, o=O, lse=None, ws=WS, ws_bytes=1 << 32):
    return lib.gdn_paged_attn(None if c is None else ctypes.byref(c), q, q_stride, o, lse, ws,
                              ws_bytes, None)


def rope(lib, c, r=None, q=Q, sq=1024, k=K, sk=256, v=V, sv=256, o=O):
    r = fake_rope() if r is None else r
    return lib.gdn_rope_append(None if c is None else ctypes.byref(c),
                               None if r is False else ctypes.byref(r), q, sq, k, sk, v, sv, o, None)


BAD = [
    (dict(batch=-1), 2), (dict(q_heads=0), 2), (dict(q_heads=7), 2), (dict(kv_heads=0), 2),
    (dict(max_T=-1), 2), (dict(max_T=65537), 2), (dict(window=-1), 2), (dict(sinks=-1), 2),
    (dict(sinks=4), 2), (dict(scale=0.0), 2), (dict(scale=-1.0), 2),
    (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(reserved=1), 2),
    (dict(max_pages=0), 2), (dict(max_pages=1 << 28), 2), (dict(n_pages=0), 2),
    (dict(n_pages=1 << 31), 2), (dict(page_stride=4095), 2), (dict(page_stride=4100), 2),
    (dict(cu_seqlens=CU, n_tok=-1), 2), (dict(cu_seqlens=CU, n_tok=1 << 31), 2),
    (dict(batch=1 << 20, max_T=65536), 2),
    (dict(dtype=2), 3),
    (dict(head_dim=96), 4), (dict(page_size=48), 4), (dict(page_size=8), 4),
    (dict(page_size=512), 4),
    (dict(k_pages=None), 1), (dict(v_pages=None), 1), (dict(page_table=None), 1),
    (dict(kv_len=None), 1),
    (dict(k_pages=BASE + 8), 7), (dict(page_table=BASE + 2 * STEP + 2), 7),
    (dict(dev_err=BASE + 4 * STEP + 1), 7),
]


@pytest.mark.parametrize("over,status", BAD)
def test_both_calls_refuse(lib, over, status):
    c = fake(**over)
    stride = max(1024, c.q_heads * c.head_dim)
    assert attn(lib, c, q_stride=stride) == status
    assert rope(lib, c, sq=stride, r=fake_rope(rot_dim=64)) == status


def test_attention_refuses(lib):
    assert attn(lib, None) == 1
    c = fake()
    assert attn(lib, c, q=None) == 1
    assert attn(lib, c, o=None) == 1
    assert attn(lib, c, ws=None) == 1
    assert attn(lib, c, q_stride=1016) == 2      # rows overlap
    assert attn(lib, c, q_stride=1028) == 2      # rows not 16-byte aligned
    assert attn(lib, c, ws_bytes=lib.gdn_paged_attn_workspace(ctypes.byref(c)) - 1) == 2
    assert attn(lib, c, q=Q + 8) == 7
    assert attn(lib, c, o=O + 4) == 7
    assert attn(lib, c, ws=WS + 8) == 7
    assert attn(lib, c, lse=LSE + 2) == 7
    assert attn(lib, c, o=Q) == 8
    assert attn(lib, c, o=c.k_pages) == 8
    assert attn(lib, c, lse=O) == 8
    assert attn(lib, c, ws=c.v_pages) == 8
    assert attn(lib, c, ws=O) == 8


def test_rope_refuses(lib):
    assert rope(lib, None) == 1
    assert rope(lib, fake(), r=False) == 1
    for over in (dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=136), dict(rot_dim=144),
                 dict(interleaved=2), dict(mscale=float("inf")), dict(reserved=1)):
        assert rope(lib, fake(), r=fake_rope(**over)) == 2, over
    assert rope(lib, fake(), r=fake_rope(inv_freq=None)) == 1
    assert rope(lib, fake(), r=fake_rope(inv_freq=BASE + 5 * STEP + 2)) == 7
    assert rope(lib, fake(), q=None) == 1
    assert rope(lib, fake(), sk=248) == 2
    assert rope(lib, fake(), sv=260) == 2
    assert rope(lib, fake(), v=V + 8) == 7
    assert rope(lib, fake(), o=Q) == 8
    assert rope(lib, fake(), o=fake().k_pages) == 8
    assert rope(lib, fake(), k=fake().k_pages) == 8     # the pages over the new keys
    assert rope(lib, fake(v_pages=BASE)) == 8           # one set of pages for both


def test_nothing_to_do(lib):
    for c in (fake(batch=0, k_pages=None), fake(max_T=0, kv_len=None),
              fake(cu_seqlens=CU, n_tok=0, page_table=None)):
        assert attn(lib, c, q=None, o=None, ws=None) == 0
        assert rope(lib, c, q=None, k=None, v=None, o=None) == 0


def test_workspace(lib):
    small = lib.gdn_paged_attn_workspace(ctypes.byref(fake(head_dim=64)))
    assert 0 < small < lib.gdn_paged_attn_workspace(ctypes.byref(fake())) < 1 << 28
    assert lib.gdn_paged_attn_workspace(ctypes.byref(fake(head_dim=96))) == -1
    assert lib.gdn_paged_attn_workspace(None) == -1


# ---------------------------------------------------------------- the binding's checks

def cpu_step(**over):
    a = dict(q_heads=4, k_pages=torch.zeros(5, 2, 16, 64), v_pages=torch.zeros(5, 2, 16, 64),
             page_table=torch.zeros(3, 2, dtype=torch.int32),
             kv_len=torch.zeros(3, dtype=torch.int32), max_T=2)
    a.update(over)
    return binding.make_attn(**a)


@pytest.mark.parametrize("over,error", [
    (dict(k_pages=torch.zeros(5, 2, 16)), ValueError),
    (dict(v_pages=torch.zeros(5, 2, 16, 32)), ValueError),
    (dict(v_pages=torch.zeros(5, 2, 16, 64, dtype=torch.bfloat16)), TypeError),
    (dict(k_pages=torch.zeros(5, 2, 16, 64).half(), v_pages=torch.zeros(5, 2, 16, 64).half()), TypeError),
    (dict(k_pages=torch.zeros(5, 16, 2, 64).transpose(1, 2)), ValueError),
    (dict(k_pages=torch.zeros(10, 2, 16, 64)[::2]), ValueError),   # page strides differ
    (dict(page_table=torch.zeros(2, 2, dtype=torch.int32)), ValueError),
    (dict(page_table=torch.zeros(3, 2)), TypeError),
    (dict(kv_len=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(cu_seqlens=torch.zeros(4, dtype=torch.int32)), ValueError),           # no n_tok
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32), n_tok=2), ValueError),
])
def test_make_attn_refuses(over, error):
    with pytest.raises(error):
        cpu_step(**over)


def test_calls_check_their_tensors():
    a = cpu_step()
    r = binding.make_rope(inv_freq=torch.ones(32))
    q, kv, o = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64), torch.zeros(6, 4, 64)
    ws = torch.zeros(16, dtype=torch.uint8)
    for bad in (torch.zeros(5, 4, 64), torch.zeros(6, 4, 32), torch.zeros(6, 64, 4).transpose(1, 2)):
        with pytest.raises(ValueError):
            binding.gdn_paged_attn(a, bad, o, workspace=ws)
        with pytest.raises(ValueError):
            binding.gdn_rope_append(a, r, bad, kv, kv, o)
    with pytest.raises(TypeError):
        binding.gdn_paged_attn(a, q.bfloat16(), o, workspace=ws)
    with pytest.raises(ValueError):
        binding.gdn_paged_attn(a, q, torch.zeros(6, 8, 64)[:, :4], workspace=ws)
    with pytest.raises(ValueError):
        binding.gdn_paged_attn(a, q, o, lse=torch.zeros(6, 3), workspace=ws)
    with pytest.raises(ValueError):
        binding.gdn_rope_append(a, binding.make_rope(inv_freq=torch.ones(32), positions=torch.zeros(
            5, dtype=torch.int32)), q, kv, kv, o)
    with pytest.raises(TypeError):
        binding.make_rope(inv_freq=torch.ones(32).double())
