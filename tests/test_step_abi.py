"""Linear attention, sampled acceptance and page planning without a GPU: struct layouts, what the
host validation refuses before any CUDA call, and what the binding's own checks refuse."""
import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decode_gated_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, STEP = 1 << 44, 1 << 40


def at(i):
    return BASE + i * STEP


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        import speculative_decode_gated_gb300 as pkg
        pkg.build()
    return binding.lib()


@pytest.mark.parametrize("cls", [binding.gdn_linear, binding.gdn_sample, binding.gdn_pages])
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


# ---------------------------------------------------------------- linear attention

def linear(**over):
    """A step with plausible, aligned fake device addresses (never dereferenced)."""
    c = binding.gdn_linear()
    c.batch, c.heads, c.k_heads, c.dk, c.dv, c.max_T = 2, 8, 4, 128, 64, 4
    c.dtype, c.scale, c.n_tok = binding.GDN_BF16, 1.0, 8
    c.q, c.k, c.v, c.log_decay, c.pool, c.slot_ids = (at(i) for i in range(6))
    c.q_stride, c.k_stride, c.v_stride, c.decay_stride, c.pool_slots = 512, 512, 512, 8, 3
    for k, v in over.items():
        setattr(c, k, v)
    return c


O, ACC = at(20), at(21)
LINEAR_BAD = [
    (dict(batch=-1), 2), (dict(heads=0), 2), (dict(k_heads=0), 2), (dict(k_heads=3), 2),
    (dict(max_T=-1), 2), (dict(max_T=65537), 2), (dict(scale=float("nan")), 2),
    (dict(scale=float("inf")), 2), (dict(cu_seqlens=at(6), n_tok=-1), 2),
    (dict(cu_seqlens=at(6), n_tok=1 << 31), 2), (dict(batch=1 << 28), 2),
    (dict(batch=1 << 20, max_T=4096, pool_slots=1 << 20), 2), (dict(pool_slots=1), 2),
    (dict(k_stride=511), 2), (dict(k_stride=516), 2), (dict(v_stride=504), 2),
    (dict(k_stride=(1 << 36) + 8), 2), (dict(decay_stride=7), 2), (dict(decay_stride=-1), 2),
    (dict(dtype=2), 3), (dict(dk=96), 4), (dict(dk=512), 4), (dict(dv=48), 4), (dict(dv=288), 4),
    (dict(dv=0), 4),
    (dict(k=None), 1), (dict(v=None), 1), (dict(log_decay=None), 1), (dict(pool=None), 1),
    (dict(slot_ids=None), 1),
    (dict(k=at(1) + 8), 7), (dict(v=at(2) + 2), 7), (dict(log_decay=at(3) + 2), 7),
    (dict(pool=at(4) + 4), 7), (dict(slot_ids=at(5) + 1), 7), (dict(dev_err=at(7) + 2), 7),
]


@pytest.mark.parametrize("over,status", LINEAR_BAD)
def test_linear_calls_refuse(lib, over, status):
    c = ctypes.byref(linear(**over))
    assert lib.gdn_linear_verify(c, O, None) == status
    assert lib.gdn_linear_commit(c, ACC, None) == status
    assert lib.gdn_linear_step(c, O, None) == status


def test_linear_outputs_refuse(lib):
    c = linear()
    ref = ctypes.byref(c)
    for fn in (lib.gdn_linear_verify, lib.gdn_linear_step):
        assert fn(None, O, None) == 1
        assert fn(ref, None, None) == 1
        assert fn(ref, O + 8, None) == 7
        for x in (c.q, c.k, c.v, c.log_decay, c.pool, c.slot_ids):
            assert fn(ref, x, None) == 8
        assert fn(ctypes.byref(linear(q=None)), O, None) == 1
        assert fn(ctypes.byref(linear(q=at(0) + 8)), O, None) == 7
        assert fn(ctypes.byref(linear(q_stride=8)), O, None) == 2
    assert lib.gdn_linear_commit(ref, None, None) == 1
    assert lib.gdn_linear_commit(ref, ACC + 2, None) == 7
    assert lib.gdn_linear_commit(ref, c.pool, None) == 8
    # a pool over the rows: refused by the calls that write it
    over = ctypes.byref(linear(pool=at(1)))
    assert lib.gdn_linear_commit(over, ACC, None) == 8
    assert lib.gdn_linear_step(over, O, None) == 8


def test_linear_nothing_to_do(lib):
    for over in (dict(batch=0), dict(max_T=0), dict(cu_seqlens=at(6), n_tok=0)):
        c = ctypes.byref(linear(**over))
        assert lib.gdn_linear_verify(c, O, None) == 0
        assert lib.gdn_linear_commit(c, ACC, None) == 0
        assert lib.gdn_linear_step(c, O, None) == 0


def rows(n, *shape, dtype=torch.bfloat16):
    return torch.zeros((n,) + shape, dtype=dtype)


def linear_tensors(**over):
    t = dict(q=rows(8, 4, 64), k=rows(8, 4, 64), v=rows(8, 8, 32), log_decay=torch.zeros(8, 8),
             pool=torch.zeros(3, 8, 64, 32), slot_ids=torch.zeros(2, dtype=torch.int32), max_T=4)
    t.update(over)
    return t


@pytest.mark.parametrize("over,error", [
    (dict(k=rows(8, 4, 64, dtype=torch.float16)), TypeError),
    (dict(v=rows(8, 8, 32, dtype=torch.float32)), TypeError),
    (dict(q=rows(8, 4, 64, dtype=torch.float32)), TypeError),
    (dict(log_decay=torch.zeros(8, 8, dtype=torch.float64)), TypeError),
    (dict(slot_ids=torch.zeros(2)), TypeError),
    (dict(pool=torch.zeros(3, 8, 64)), ValueError), (dict(max_T=5), ValueError),
    (dict(k=rows(8, 4, 32)), ValueError), (dict(q=rows(8, 2, 64)), ValueError),
    (dict(v=rows(7, 8, 32)), ValueError), (dict(k=rows(8, 64, 4).transpose(1, 2)), ValueError),
    (dict(log_decay=torch.zeros(7, 8)), ValueError), (dict(log_decay=torch.zeros(16)[::2]), ValueError),
    (dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(k=torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="meta")), ValueError),
])
def test_make_linear_refuses(over, error):
    with pytest.raises(error):
        binding.make_linear(**linear_tensors(**over))


def test_linear_strides(lib):
    wide = rows(8, 16, 64)
    lin = binding.make_linear(**linear_tensors(k=wide[:, 3:7], log_decay=torch.zeros(8)))
    assert (lin.c.k_stride, lin.c.q_stride, lin.c.v_stride, lin.c.decay_stride) == (1024, 256, 256, 0)
    assert lin.c.k == wide.data_ptr() + 3 * 64 * 2
    # rows that an expand() made the same are constants; a single row is one
    assert binding.make_linear(**linear_tensors(log_decay=torch.zeros(1, 8).expand(8, 8))).c.decay_stride == 0
    o = rows(8, 8, 32)
    with pytest.raises(ValueError):  # tensors of the host
        binding.gdn_linear_step(lin, o)
    for bad in (rows(8, 8, 64), rows(8, 32, 8).transpose(1, 2)):
        with pytest.raises(ValueError):
            binding.gdn_linear_step(lin, bad)
    with pytest.raises(TypeError):
        binding.gdn_linear_verify(lin, o.float())
    with pytest.raises(ValueError):
        binding.gdn_linear_commit(lin, torch.zeros(3, dtype=torch.int32))


# ---------------------------------------------------------------- sampled drafts

def sample(**over):
    c = binding.gdn_sample()
    c.batch, c.max_T, c.vocab, c.n_tok = 2, 4, 100, 8
    c.draft_ids, c.target_probs, c.draft_probs, c.u_accept, c.u_sample = (at(i) for i in range(5))
    c.target_stride = c.draft_stride = 100
    for k, v in over.items():
        setattr(c, k, v)
    return c


NEXT = at(22)


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), 2), (dict(max_T=-1), 2), (dict(max_T=1025), 2), (dict(vocab=0), 2),
    (dict(vocab=262145), 2), (dict(reserved=1), 2), (dict(target_stride=99), 2),
    (dict(draft_stride=99), 2), (dict(target_stride=(1 << 36) + 1), 2),
    (dict(cu_seqlens=at(6), n_tok=-1), 2), (dict(cu_seqlens=at(6), n_tok=1 << 31), 2),
    (dict(batch=1 << 28), 2),
    (dict(draft_ids=None), 1), (dict(target_probs=None), 1), (dict(u_accept=None), 1),
    (dict(u_sample=None), 1),
    (dict(draft_ids=at(0) + 1), 7), (dict(target_probs=at(1) + 2), 7), (dict(draft_probs=at(2) + 2), 7),
    (dict(u_accept=at(3) + 2), 7), (dict(u_sample=at(4) + 2), 7), (dict(cu_seqlens=at(6) + 2), 7),
    (dict(dev_err=at(7) + 2), 7),
    (dict(u_sample=ACC), 8), (dict(draft_ids=NEXT), 8), (dict(dev_err=ACC), 8),
])
def test_accept_sample_refuses(lib, over, status):
    assert lib.gdn_accept_sample(ctypes.byref(sample(**over)), ACC, NEXT, None) == status


def test_accept_sample_outputs_refuse(lib):
    c = ctypes.byref(sample())
    assert lib.gdn_accept_sample(None, ACC, NEXT, None) == 1
    assert lib.gdn_accept_sample(c, None, NEXT, None) == 1
    assert lib.gdn_accept_sample(c, ACC, None, None) == 1
    assert lib.gdn_accept_sample(c, ACC + 2, NEXT, None) == 7
    assert lib.gdn_accept_sample(c, ACC, ACC + 4, None) == 8
    assert lib.gdn_accept_sample(ctypes.byref(sample(batch=0)), None, None, None) == 0


@pytest.mark.parametrize("over,error", [
    (dict(target_probs=torch.zeros(8, 10, dtype=torch.bfloat16)), TypeError),
    (dict(draft_ids=torch.zeros(8, dtype=torch.int64)), TypeError),
    (dict(u_accept=torch.zeros(8, dtype=torch.float64)), TypeError),
    (dict(target_probs=torch.zeros(7, 10)), ValueError), (dict(u_accept=torch.zeros(7)), ValueError),
    (dict(draft_probs=torch.zeros(8, 11)), ValueError), (dict(max_T=3), ValueError),
    (dict(target_probs=torch.zeros(10, 8).t()), ValueError),
    (dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), ValueError),
])
def test_make_sample_refuses(over, error):
    t = dict(draft_ids=torch.zeros(8, dtype=torch.int32), target_probs=torch.zeros(8, 10),
             u_accept=torch.zeros(8), u_sample=torch.zeros(2), max_T=4)
    binding.make_sample(**t)
    t.update(over)
    with pytest.raises(error):
        binding.make_sample(**t)


# ---------------------------------------------------------------- pages

def pages(**over):
    c = binding.gdn_pages()
    c.batch, c.max_T, c.page_size, c.max_pages, c.n_pages, c.max_rows = 4, 16, 16, 10, 50, 64
    (c.rows, c.accepted, c.done, c.kv_len, c.held, c.free_count, c.free_pages, c.page_table,
     c.cu_seqlens, c.slots, c.positions) = (at(i) for i in range(11))
    c.kv_len_out, c.held_out, c.free_count_out = c.kv_len, c.held, c.free_count
    for k, v in over.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("over,status", [
    (dict(batch=-1), 2), (dict(max_T=-1), 2), (dict(max_T=65537), 2), (dict(max_pages=0), 2),
    (dict(n_pages=0), 2), (dict(n_pages=1 << 31), 2), (dict(max_rows=-1), 2),
    (dict(max_pages=1 << 28), 2), (dict(batch=1 << 28), 2), (dict(batch=1 << 20, max_T=4096), 2),
    (dict(page_size=8), 4), (dict(page_size=48), 4), (dict(page_size=512), 4),
    (dict(kv_len=None), 1), (dict(held=None), 1), (dict(free_count=None), 1),
    (dict(kv_len_out=None), 1), (dict(held_out=None), 1), (dict(free_count_out=None), 1),
    (dict(free_pages=None), 1), (dict(page_table=None), 1), (dict(cu_seqlens=None), 1),
    (dict(rows=at(0) + 2), 7), (dict(slots=at(9) + 4), 7), (dict(positions=at(10) + 2), 7),
    (dict(page_table=at(7) + 2), 7), (dict(dev_err=at(11) + 2), 7),
    (dict(kv_len_out=at(3) + 4), 8), (dict(held_out=at(3)), 8), (dict(free_count_out=at(3)), 8),
    (dict(cu_seqlens=at(0)), 8), (dict(page_table=at(6)), 8), (dict(positions=at(1)), 8),
    (dict(slots=at(10)), 8), (dict(dev_err=at(2)), 8),
])
def test_plan_pages_refuses(lib, over, status):
    assert lib.gdn_plan_pages(ctypes.byref(pages(**over)), None) == status
    assert lib.gdn_plan_pages(None, None) == 1
    assert lib.gdn_plan_pages(ctypes.byref(pages(batch=0)), None) == 0


@pytest.mark.parametrize("over,error", [
    (dict(kv_len=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(rows=torch.zeros(5, dtype=torch.int32)), ValueError),
    (dict(cu_seqlens=torch.zeros(4, dtype=torch.int32)), ValueError),
    (dict(free_count=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(page_table=torch.zeros(40, dtype=torch.int32)), ValueError),
    (dict(slots=torch.zeros(4, dtype=torch.int64), positions=torch.zeros(5, dtype=torch.int32)), ValueError),
    (dict(slots=torch.zeros(4, dtype=torch.int32)), TypeError),
    (dict(held=torch.zeros(4, dtype=torch.int64)), TypeError),
])
def test_make_pages_refuses(over, error):
    def i(*n):
        return torch.zeros(n, dtype=torch.int32)
    t = dict(page_table=i(4, 10), page_size=16, max_T=16, kv_len=i(4), held=i(4), free_pages=i(50),
             free_count=i(1), cu_seqlens=i(5))
    p = binding.make_pages(**t)
    assert (p.c.kv_len_out, p.c.held_out, p.c.free_count_out) == (p.c.kv_len, p.c.held, p.c.free_count)
    t.update(over)
    with pytest.raises(error):
        binding.make_pages(**t)


def test_read_error_refuses(lib):
    code = ctypes.c_int32(-1)
    assert lib.gdn_read_error(None, None, ctypes.byref(code)) == 0 and code.value == 0
    assert lib.gdn_read_error(at(0), None, None) == 1
    with pytest.raises(ValueError):
        binding.gdn_read_error(torch.zeros(1, dtype=torch.int32))
