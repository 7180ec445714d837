"""A speculative step with sampled drafts (gdn_plan_pages, gdn_linear_verify, gdn_accept_sample,
gdn_linear_commit) as one captured graph, in bfloat16 with heads that the tensor-core kernels take: drafts of up to 6 and 20 rows,
and of up to 50, which the prompts' kernel takes.

Whole numbers have to equal the oracles'.  Outputs and states are held to the oracle from the states before each
step, by the terms of test_linear_drafts_gpu.py: (5 n + dk + 8) 2^-24 of the terms' absolute values for n
rows; 2^-17 of them for the two bfloat16 terms of states and weights in a verify (2^-8 in the
prompts' kernel), 2^-17 for what the prompts' kernel adds to a state; and a bfloat16 output's own 2^-8."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu

B, H, HK, DV, VOCAB, PAGE, WIDTH, N_PAGES = 4, 4, 2, 128, 211, 16, 24, 90


@pytest.mark.parametrize("dk,T", [(128, 6), (64, 20), (128, 50)])
def test_steps_in_a_graph(dk, T):
    rng = np.random.default_rng(dk + T)
    n = B * T

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def zeros(*shape, dtype=torch.float32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    bf = torch.bfloat16
    q, k, v = zeros(n, HK, dk, dtype=bf), zeros(n, HK, dk, dtype=bf), zeros(n, H, DV, dtype=bf)
    g, o = zeros(n, H), zeros(n, H, DV, dtype=bf)
    pool = torch.from_numpy(rng.standard_normal((B + 1, H, dk, DV)).astype(np.float32)).cuda()
    slots = rng.permutation(B + 1)[:B]
    free = [int(x) for x in rng.permutation(N_PAGES)]
    kv_len, held, table, last = [0] * B, [0] * B, [[-1] * WIDTH for _ in range(B)], [0] * B
    d_len, d_held, cu = i32(kv_len), i32(held), i32([0] * (B + 1))
    rows, accepted, nxt = i32([0] * B), i32([0] * B), i32([0] * B)
    d_slots, d_pos, ids, err = zeros(n, dtype=torch.int64), i32([0] * n), i32([0] * n), i32([0])
    p, draft, u, us = zeros(n, VOCAB), zeros(n, VOCAB), zeros(n), zeros(B)
    pages = binding.make_pages(page_table=i32(table), page_size=PAGE, max_T=T, kv_len=d_len, held=d_held,
                               free_pages=i32(free), free_count=i32([N_PAGES]), rows=rows, accepted=accepted,
                               cu_seqlens=cu, slots=d_slots, positions=d_pos, dev_err=err)
    lin = binding.make_linear(q=q, k=k, v=v, log_decay=g, pool=pool, slot_ids=i32(slots), max_T=T, cu_seqlens=cu,
                              scale=0.5, dev_err=err)
    sample = binding.make_sample(draft_ids=ids, target_probs=p, draft_probs=draft, u_accept=u, u_sample=us, max_T=T,
                                 cu_seqlens=cu, dev_err=err)

    def step():
        binding.gdn_plan_pages(pages)
        binding.gdn_linear_verify(lin, o)
        binding.gdn_accept_sample(sample, accepted, nxt)
        binding.gdn_linear_commit(lin, accepted)

    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()  # no rows yet
    stream.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()

    def softmax(x):
        e = np.exp(x - x.max(1, keepdims=True))
        return (e / e.sum(1, keepdims=True)).astype(np.float32)

    kept = 0
    for t in range(4):
        wanted = [T] + [int(rng.integers(0, T + 1)) for _ in range(B - 1)]
        logits = rng.standard_normal((n, VOCAB)) * 3
        hp, hd = softmax(logits), softmax(logits + 0.3 * rng.standard_normal((n, VOCAB)))
        hi = np.array([0] + [rng.choice(VOCAB, p=x / x.sum()) for x in hd[:-1].astype(np.float64)])
        hu, hus = rng.random(n, np.float32), rng.random(B, np.float32)
        for x, scale in ((q, 1.0), (k, dk ** -0.5), (v, 1.0)):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32) * np.float32(scale)))
        g.copy_(torch.from_numpy(-0.3 * rng.random((n, H), np.float32)))
        for x, y in ((rows, wanted), (ids, hi), (p, hp), (draft, hd), (u, hu), (us, hus)):
            x.copy_(torch.from_numpy(np.asarray(y)))
        before = pool.cpu().numpy()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        stream.synchronize()

        w = oracle.plan_pages(kv_len, held, free, table, PAGE, T, N_PAGES, wanted, last, [0] * B)
        m, off = w["cu"][-1], np.asarray(w["cu"], np.int64)
        assert int(err.item()) == w["err"] == 0 and cu.tolist() == w["cu"]
        assert d_len.tolist() == list(w["kv_len"]) and d_held.tolist() == list(w["held"])
        assert d_slots[:m].tolist() == [int(x) for x in w["slots"]]
        kv_len, held, free, table = w["kv_len"], w["held"], w["free"], w["table"]
        want_acc, want_next = oracle.accept_sample(hi[:m], hp[:m], hd[:m], hu[:m], hus, off)
        last = accepted.tolist()
        assert last == [int(x) for x in want_acc] and nxt.tolist() == [int(x) for x in want_next]
        kept += sum(a > 1 for a in last)

        host = [x[:m].float().cpu().numpy() for x in (q, k, v, g)]
        want_o, _, mag, _ = oracle.linear_attention(*host, before[slots], off, 0.5)
        _, want_s, _, size = oracle.linear_attention(*host, before[slots], off, 0.5, rows=last)
        unit = (5 * T + dk + 8) * 2.0 ** -24
        tol = (unit + (2.0 ** -8 if T >= 48 else 2.0 ** -17)) * mag
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want_o) + 1e-30
        assert np.all(np.abs(o[:m].float().cpu().numpy() - want_o) <= tol)
        after = pool.cpu().numpy()
        for r in range(B):
            if last[r]:
                limit = (unit + (2.0 ** -17 if T >= 48 else 0.0)) * size[r] + 1e-30
                assert np.all(np.abs(after[slots[r]] - want_s[r]) <= limit)
            else:
                assert np.array_equal(after[slots[r]], before[slots[r]])
    assert kept > 0
