"""A speculative step with sampled drafts as a serving loop runs it: gdn_plan_pages, gdn_linear_verify,
gdn_accept_sample and gdn_linear_commit captured in one graph, replayed with other drafts, row counts and
random numbers.  Lengths, pages, accepted rows and tokens have to equal the oracles'; outputs and
states are held to them from the states before each step (float32: every term of a sum is off by at
most (5 n + dk + 8) 2^-24 of itself, n rows: 2^-22 a decay, 8 roundings of its product, 2^-24 an
addition)."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu

B, T, H, HK, DK, DV, VOCAB, PAGE, WIDTH, N_PAGES = 5, 6, 4, 2, 64, 96, 501, 16, 8, 40


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_steps_in_a_graph(dtype):
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    rng = np.random.default_rng(0)
    n = B * T  # an upper bound of the rows

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def zeros(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    q, k, v = zeros(n, HK, DK, dtype=dt), zeros(n, HK, DK, dtype=dt), zeros(n, H, DV, dtype=dt)
    g, o = zeros(n, H), zeros(n, H, DV, dtype=dt)
    pool = torch.from_numpy(rng.standard_normal((B + 1, H, DK, DV)).astype(np.float32)).cuda()
    slots = rng.permutation(B + 1)[:B]
    free = [int(x) for x in rng.permutation(N_PAGES)]
    kv_len, held, table = [0] * B, [0] * B, [[-1] * WIDTH for _ in range(B)]
    d_len, d_held, d_table, d_free = i32(kv_len), i32(held), i32(table), i32(free)
    d_count, cu, rows, accepted, done = i32([N_PAGES]), i32([0] * (B + 1)), i32([0] * B), i32([0] * B), i32([0] * B)
    d_slots, d_pos = zeros(n, dtype=torch.int64), zeros(n, dtype=torch.int32)
    ids, nxt, err = zeros(n, dtype=torch.int32), zeros(B, dtype=torch.int32), zeros(1, dtype=torch.int32)
    p, draft, u, us = zeros(n, VOCAB), zeros(n, VOCAB), zeros(n), zeros(B)
    pages = binding.make_pages(page_table=d_table, page_size=PAGE, max_T=T, kv_len=d_len, held=d_held,
                               free_pages=d_free, free_count=d_count, rows=rows, accepted=accepted, done=done,
                               cu_seqlens=cu, slots=d_slots, positions=d_pos, dev_err=err)
    lin = binding.make_linear(q=q, k=k, v=v, log_decay=g, pool=pool, slot_ids=i32(slots), max_T=T,
                              cu_seqlens=cu, scale=0.5, dev_err=err)
    sample = binding.make_sample(draft_ids=ids, target_probs=p, draft_probs=draft, u_accept=u, u_sample=us,
                                 max_T=T, cu_seqlens=cu, dev_err=err)

    def step():
        binding.gdn_plan_pages(pages)
        binding.gdn_linear_verify(lin, o)
        binding.gdn_accept_sample(sample, accepted, nxt)
        binding.gdn_linear_commit(lin, accepted)

    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        step()  # no rows yet
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()

    def softmax(x):
        e = np.exp(x - x.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True)).astype(np.float32)

    last = [0] * B
    kept_any = 0
    for t in range(5):
        wanted = [int(rng.integers(0, T + 1)) for _ in range(B)]
        over = [int(t == 3 and r == 1) for r in range(B)]
        logits = rng.standard_normal((n, VOCAB)) * 3
        hp, hd = softmax(logits), softmax(logits + 0.5 * rng.standard_normal((n, VOCAB)))
        hi = np.zeros(n, np.int64)
        for i in range(1, n):
            c = np.cumsum(hd[i - 1], dtype=np.float64)
            hi[i] = min(int(np.searchsorted(c, rng.random() * c[-1])), VOCAB - 1)
        hu, hus = rng.random(n, np.float32), rng.random(B, np.float32)
        for x, scale in ((q, 1.0), (k, DK ** -0.5), (v, 1.0)):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32) * np.float32(scale)))
        g.copy_(torch.from_numpy(-0.3 * rng.random((n, H), np.float32)))
        for x, y in ((rows, wanted), (done, over), (ids, hi), (p, hp), (draft, hd), (u, hu), (us, hus)):
            x.copy_(torch.from_numpy(np.asarray(y)))
        before = pool.cpu().numpy()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()

        w = oracle.plan_pages(kv_len, held, free, table, PAGE, T, N_PAGES, wanted, last, over)
        assert int(err.item()) == w["err"] == 0
        assert cu.tolist() == w["cu"]
        m = w["cu"][-1]
        assert d_len.tolist() == list(w["kv_len"]) and d_held.tolist() == list(w["held"])
        assert d_slots[:m].tolist() == [int(x) for x in w["slots"]]
        assert d_pos[:m].tolist() == [int(x) for x in w["positions"]]
        kv_len, held, free, table = w["kv_len"], w["held"], w["free"], w["table"]

        off = np.asarray(w["cu"], np.int64)
        want_acc, want_next = oracle.accept_sample(hi[:m], hp[:m], hd[:m], hu[:m], hus, off)
        last = accepted.tolist()
        assert last == [int(x) for x in want_acc]
        assert nxt.tolist() == [int(x) for x in want_next]
        kept_any += sum(a > 1 for a in last)

        host = [x[:m].float().cpu().numpy() for x in (q, k, v, g)]
        want_o, _, mag, _ = oracle.linear_attention(*host, before[slots], off, 0.5)
        _, want_s, _, mag_s = oracle.linear_attention(*host, before[slots], off, 0.5, rows=last)
        unit = (5 * T + DK + 8) * 2.0 ** -24
        tol = unit * mag + 1e-30
        if dtype == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want_o)
        assert np.all(np.abs(o[:m].float().cpu().numpy() - want_o) <= tol)
        after = pool.cpu().numpy()
        for r in range(B):
            if last[r]:
                assert np.all(np.abs(after[slots[r]] - want_s[r]) <= unit * mag_s[r] + 1e-30)
            else:
                assert np.array_equal(after[slots[r]], before[slots[r]])
        other = [s for s in range(B + 1) if s not in slots]
        assert np.array_equal(after[other], before[other])
    assert kept_any > 0
