"""GPU parity of attention over the paged cache against the float64 oracle: every
type, head layout and page size, one row to several hundred, contexts around the tiles'
and pages' ends, windows with sinks, and caches whose unseen places hold NaN."""
import numpy as np
import pytest
import torch

from attn_cases import Case, to_dev
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd", [32, 64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (8, 2), (15, 3), (16, 1), (40, 2)])
def test_head_layouts(dtype, hd, heads):
    Case(new=[1, 3, 0, 2], old=[40, 0, 9, 131], q_heads=heads[0], kv_heads=heads[1], hd=hd,
         dtype=dtype, seed=hd + heads[0]).device().run().check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T", [1, 16, 70])
def test_pages(page, hd, T):
    Case(new=[T, T], old=[page - 1, 5 * page + 3], q_heads=8, kv_heads=2, hd=hd, page=page,
         seed=page + T).device().run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("old", [0, 1, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 256, 1000])
@pytest.mark.parametrize("T", [1, 2, 16])
def test_context_lengths(dtype, old, T):
    Case(new=[T], old=[old], q_heads=4, kv_heads=2, hd=64, dtype=dtype,
         seed=old).device(ragged=False).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,G,hd", [(17, 1, 64), (100, 4, 128), (129, 1, 128), (257, 2, 64),
                                    (300, 5, 32), (64, 8, 256), (33, 16, 128)])
def test_prompt_chunks(dtype, T, G, hd):
    Case(new=[T, 1, T // 2], old=[0, 200, 77], q_heads=2 * G, kv_heads=2, hd=hd, page=32,
         dtype=dtype, seed=T).device().run().check()


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp32", 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 0), (64, 3), (100, 20),
                                          (128, 130), (300, 1), (100000, 4)])
@pytest.mark.parametrize("T", [1, 16, 150])
def test_windows(dtype, hd, window, sinks, T):
    Case(new=[T, T // 2, 1], old=[411, 130, 3], q_heads=4, kv_heads=2, hd=hd, window=window,
         sinks=sinks, dtype=dtype, seed=window + T).device().run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 16, 90])
@pytest.mark.parametrize("fill", [np.inf, -np.inf, 3e38, -3e38])
def test_unseen_places_hold_anything(dtype, T, fill):
    Case(new=[T, T], old=[90, 301], q_heads=8, kv_heads=2, hd=128, window=70, sinks=2, page=32,
         dtype=dtype, fill=fill, seed=T).device().run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,T,G", [(64, 16, 1), (128, 16, 4), (128, 200, 2), (256, 9, 2)])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_bad_token_reaches_only_the_rows_that_see_it(dtype, hd, T, G, what, value):
    c = Case(new=[T], old=[37], q_heads=2 * G, kv_heads=2, hd=hd, dtype=dtype, seed=T)
    bad = T // 2  # a draft whose key or value is not finite, at one element of one head
    at = c.table[0, (37 + bad) // 16], 1, (37 + bad) % 16, 3
    (c.k if what == "k" else c.v)[at] = value
    c.device().run()
    clean = np.arange(T) < bad
    c.check(rows=clean)                      # rows before it
    got = c.o.float().cpu().numpy()
    assert np.all(np.isfinite(got[:, :G]))   # the other key head
    if what == "v":
        assert not np.any(np.isfinite(got[~clean][:, G:, 3]))
        assert np.all(np.isfinite(got[:, G:, [0, 1, 2, 4]]))
    elif np.isnan(value):
        assert np.all(np.isnan(got[~clean][:, G:]))


@pytest.mark.parametrize("T", [1, 16, 100])
def test_a_bad_token_that_leaves_the_window(T):
    c = Case(new=[T], old=[150], q_heads=4, kv_heads=2, hd=128, window=40, seed=T)
    first = 150 - 40 + 1  # the first place that the first row sees, and no other row
    c.v[c.table[0, first // 16], :, first % 16] = np.inf
    c.device().run()
    got = c.o.float().cpu().numpy()
    assert not np.any(np.isfinite(got[0]))
    c.check(rows=np.arange(T) > 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 40])
def test_large_scores(dtype, T):
    # scores of some hundred units: one place takes all the weight, the rest underflow
    c = Case(new=[T], old=[333], q_heads=4, kv_heads=1, hd=64, dtype=dtype, qscale=40.0, seed=T)
    c.device().run()
    o, lse, mean = c.expected()
    # the score's error grows with the score: 64 products of a few hundred, in float32
    tol = 2.0 ** -8 * (np.abs(o) + mean) + 2.0 ** -6 * mean
    assert np.all(np.abs(c.o.float().cpu().numpy() - o) <= tol)
    assert np.all(np.abs(c.lse.cpu().numpy() - lse) <= 2.0 ** -18 * np.abs(lse) + 2.0 ** -7)


@pytest.mark.parametrize("T", [1, 16, 130])
def test_rows_of_a_wider_projection_and_interleaved_pages(T):
    c = Case(new=[T, T], old=[100, 33], q_heads=8, kv_heads=2, hd=128, seed=T)
    c.device(interleave=True)
    wide = torch.full((c.n_tok, 12, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = to_dev(c.q, "bf16")
    c.run(q=wide[:, 2:10]).check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 16, 100])
def test_repeatable_and_without_lse(dtype, T):
    c = Case(new=[T] * 5, old=[7, 900, 40, 2500, 1], q_heads=8, kv_heads=2, hd=64, dtype=dtype,
             seed=T).device()
    a = c.run().o.clone()
    ws = c.ws
    assert not ws[9728:16384].any()              # the counters are back at zero
    ws[16384:].view(torch.float32).fill_(float("nan"))  # nothing else a call left is read by the next
    assert torch.equal(c.run(workspace=ws).o, a)
    assert torch.equal(c.run(lse=False, workspace=ws).o, a)


@pytest.mark.parametrize("dtype,kv_heads,T", [("bf16", 1, 1), ("bf16", 2, 3), ("bf16", 8, 1),
                                              ("fp32", 1, 1), ("fp32", 8, 2), ("bf16", 1, 20)])
def test_one_long_request_among_short_ones(dtype, kv_heads, T):
    # a unit of many partials: joined by the last block to write one, or by a launch of its own
    Case(new=[T, 1, T], old=[9, 20011, 300], q_heads=2 * kv_heads, kv_heads=kv_heads, hd=64,
         dtype=dtype, page=64, seed=kv_heads).device().run().check()


def test_ragged_and_uniform_rows_agree():
    c = Case(new=[16] * 6, old=[10, 300, 77, 128, 0, 64], q_heads=8, kv_heads=2, hd=128, seed=1)
    a = c.device(ragged=True).run().o.clone()
    assert torch.equal(c.device(ragged=False).run().o, a)


@pytest.mark.parametrize("T", [1, 16, 64])
def test_bad_requests_are_skipped_and_flagged(T):
    c = Case(new=[T] * 4, old=[20, 30, 40, 50], q_heads=4, kv_heads=2, hd=64, seed=3).device()
    c.dlen[1] = -1
    c.dlen[2] = c.width * c.page - T + 1
    c.run()
    assert int(c.derr.item()) == binding.GDN_DEVERR_KV_LEN
    assert torch.all(c.o[T:3 * T] == 7) and torch.all(c.lse[T:3 * T] == 7)
    c.derr.zero_()
    keep = np.r_[0:T, 3 * T:4 * T]
    c.check(rows=keep)
    c.dlen.copy_(torch.tensor(c.old, dtype=torch.int32))
    c.dcu[4] = 5 * T  # past the rows
    c.run()
    assert int(c.derr.item()) == binding.GDN_DEVERR_SEQLEN
    assert torch.all(c.o[3 * T:] == 7)
    c.derr.zero_()
    c.check(rows=np.arange(3 * T))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 16, 64])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_a_bad_page_reads_as_zeros_and_is_flagged(dtype, T, bad):
    c = Case(new=[T], old=[100], q_heads=4, kv_heads=2, hd=64, dtype=dtype, seed=3).device()
    c.dtable[0, 2] = bad
    page = c.table[0, 2]
    c.run()
    assert int(c.derr.item()) == binding.GDN_DEVERR_PAGE
    c.derr.zero_()
    c.k[page] = 0
    c.v[page] = 0
    c.check()


@pytest.mark.parametrize("dtype,hd,T", [("bf16", 128, 1), ("bf16", 128, 16), ("bf16", 64, 100),
                                        ("bf16", 256, 2), ("fp32", 128, 2)])
def test_cache_of_more_than_2_31_elements(dtype, hd, T):
    c = Case(new=[T, T], old=[70, 150], q_heads=8, kv_heads=2, hd=hd, seed=hd + T, dtype=dtype)
    c.device()
    page = 2 * 16 * hd
    n = (1 << 32) // page + 50  # elements beyond 2^32
    small, moved = (c.dk, c.dv), []
    for t in small:
        big = torch.full((n,) + t.shape[1:], float("nan"), dtype=t.dtype, device="cuda")
        big[n - t.shape[0]:] = t
        moved.append(big)
    table = torch.where(c.dtable >= 0, c.dtable + (n - c.n_pages), c.dtable)
    c.attn = binding.make_attn(q_heads=8, k_pages=moved[0], v_pages=moved[1], page_table=table,
                               kv_len=c.dlen, max_T=T, cu_seqlens=c.dcu, n_tok=c.n_tok,
                               scale=c.scale, dev_err=c.derr)
    c.run().check()


@pytest.mark.parametrize("T", [1, 16, 100])
def test_streams_and_graphs(T):
    cases = [Case(new=[T] * 3, old=[500, 40, 129], q_heads=8, kv_heads=2, hd=128,
                  seed=s).device() for s in range(2)]
    want = [c.run().o.clone() for c in cases]
    qs = [to_dev(c.q, c.dtype) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, q, s in zip(cases, qs, streams):
            binding.gdn_paged_attn(c.attn, q, c.o, lse=c.lse, workspace=c.ws, stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.o, w)
        c.o.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, q in zip(cases, qs):
            binding.gdn_paged_attn(c.attn, q, c.o, lse=c.lse, workspace=c.ws)
    for _ in range(2):
        for c in cases:
            c.o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.o, w)


def test_many_requests_of_uneven_lengths():
    rng = np.random.default_rng(9)
    new = rng.integers(0, 17, 200)
    new[7] = 16
    old = rng.integers(0, 400, 200)
    Case(new=new.tolist(), old=old.tolist(), q_heads=8, kv_heads=4, hd=64, seed=5).device().run().check()
