"""Acceptance of sampled drafts (gdn_accept_sample) against the oracle of whole numbers: every
result has to be equal."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, *, new, vocab, seed=0, lookup=False, ragged=True, pad=0, offset=0, noise=0.6, spread=3.0):
        rng = np.random.default_rng(seed)
        self.new, self.B, self.vocab = list(new), len(new), vocab
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        n = int(self.cu[-1])
        logits = rng.standard_normal((n, vocab)) * spread

        def softmax(x):
            e = np.exp(x - x.max(1, keepdims=True)) if n else x
            return (e / e.sum(1, keepdims=True)).astype(np.float32)

        self.p = softmax(logits)
        self.q = None if lookup else softmax(logits + noise * rng.standard_normal((n, vocab)))
        src = self.p if lookup else self.q
        self.ids = np.zeros(n, np.int64)
        for i in range(1, n):
            c = np.cumsum(src[i - 1], dtype=np.float64)
            self.ids[i] = min(int(np.searchsorted(c, rng.random() * c[-1])), vocab - 1)
        self.u, self.us = rng.random(n, np.float32), rng.random(self.B, np.float32)
        self.ragged, self.pad, self.offset = ragged, pad, offset
        self.max_T = max(self.new + [0])

    def run(self, **over):
        def probs(x):  # rows `pad` apart from each other, `offset` elements from the allocation's start
            if x is None:
                return None
            flat = torch.full((x.shape[0] * (self.vocab + self.pad) + self.offset + 1,), float("nan"), device="cuda")
            y = flat[self.offset:self.offset + x.shape[0] * (self.vocab + self.pad)]
            y = y.view(x.shape[0], self.vocab + self.pad)[:, :self.vocab]
            y.copy_(torch.from_numpy(x))
            return y
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        cu = torch.from_numpy(self.cu.astype(np.int32)).cuda() if self.ragged else None
        kw = dict(draft_ids=torch.from_numpy(self.ids.astype(np.int32)).cuda(), target_probs=probs(self.p),
                  draft_probs=probs(self.q), u_accept=torch.from_numpy(self.u).cuda(),
                  u_sample=torch.from_numpy(self.us).cuda(), max_T=self.max_T, cu_seqlens=cu, dev_err=self.err)
        kw.update(over)
        self.sample = binding.make_sample(**kw)
        self.acc, self.nxt = (torch.full((self.B,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
        binding.gdn_accept_sample(self.sample, self.acc, self.nxt)
        torch.cuda.synchronize()
        return self.acc.cpu().numpy(), self.nxt.cpu().numpy()

    def check(self, **over):
        acc, nxt = self.run(**over)
        want_acc, want_nxt = oracle.accept_sample(self.ids, self.p, self.q, self.u, self.us, self.cu)
        assert np.array_equal(acc, want_acc)
        assert np.array_equal(nxt, want_nxt)
        return acc


@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 33, 1000, 4097, 20011])
def test_ragged(vocab, lookup):
    c = Case(new=[1, 5, 0, 4, 8, 2, 3], vocab=vocab, lookup=lookup, seed=vocab)
    c.check()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 0), (4, 4), (0, 1), (5, 3)])
@pytest.mark.parametrize("lookup", [False, True])
def test_strides_and_alignments(pad, offset, lookup):
    Case(new=[4] * 6, vocab=5000, pad=pad, offset=offset, ragged=False, lookup=lookup, seed=1).check()


@pytest.mark.parametrize("batch,vocab", [(1, 100003), (3, 128000), (1, 262144), (700, 500)])
def test_clusters_of_every_size(batch, vocab):
    Case(new=[3] * batch, vocab=vocab, seed=2).check()


def test_long_drafts():
    # many windows of 32 rows; drafts that almost always stay
    c = Case(new=[200, 33, 34, 1, 65], vocab=50, noise=0.02, seed=3)
    acc = c.check()
    assert acc.max() > 33


def test_all_stay_or_none():
    c = Case(new=[6] * 4, vocab=300, seed=4)
    c.u[:] = 0.0
    assert set(c.check()) == {6}
    c.u[:] = np.float32(1 - 2.0 ** -24)
    c.q, c.p = np.full_like(c.q, 1.0), np.minimum(c.p, 0.5)
    assert set(c.check()) == {1}


def test_equal_distributions():
    # u q < p with q = p: every draft that has a probability stays; then the next token is p's own
    c = Case(new=[5] * 8, vocab=400, seed=5)
    c.q = c.p.copy()
    assert set(c.check()) == {5}


def test_p_nowhere_above_q_falls_back_to_p():
    c = Case(new=[3] * 8, vocab=260, seed=6)
    c.q = np.minimum(c.p * np.float32(1.5), 1)  # not normalised: what max(p - q, 0) leaves is nothing
    c.u[:] = np.float32(0.99)
    assert set(c.check()) == {1}


@pytest.mark.parametrize("us", [0.0, 1.0 - 2.0 ** -24, 2.0 ** -33, -3.0, 1.0, 5.0, float("nan"), float("inf")])
def test_ends_of_the_random_numbers(us):
    c = Case(new=[2] * 3, vocab=1500, seed=7)
    c.p[:, :40] = 0.0
    c.p[:, -40:] = 0.0
    c.us[:] = np.float32(us)
    if not np.isfinite(us):
        c.us[:] = us
        acc, nxt = c.run()
        c.us[:] = 0.0 if np.isnan(us) else 1.0
        want = oracle.accept_sample(c.ids, c.p, c.q, c.u, c.us, c.cu)
        assert np.array_equal(acc, want[0]) and np.array_equal(nxt, want[1])
    else:
        c.check()


def test_tiny_probabilities():
    # below the unit of 2^-44 nothing is drawn; denormals and 2^-44 itself
    c = Case(new=[1] * 4, vocab=70, seed=8)
    c.p[:] = 1e-40
    c.p[:, 11] = 2.0 ** -44
    c.p[:, 69] = 2.0 ** -44
    c.us = np.float32([0.0, 0.499, 0.5, 0.999])
    c.check()
    assert c.nxt.tolist() == [11, 11, 69, 69]


def test_values_that_are_no_probabilities():
    c = Case(new=[2] * 4, vocab=90, seed=9)
    c.p[:, 5], c.p[:, 6], c.p[:, 7], c.p[:, 8] = np.nan, -1.0, 3.0, np.inf
    c.q[:, 9], c.q[:, 10], c.q[:, 7] = np.nan, -np.inf, 0.25
    c.check()


def test_drafts_outside_the_vocabulary():
    for lookup in (False, True):
        c = Case(new=[3] * 4, vocab=120, seed=10, lookup=lookup)
        c.u[:] = 0.0
        c.ids[[1, 4, 8]] = [120, -1, 1 << 30]
        acc = c.check()
        assert acc.tolist() == [1, 1, 2, 3]
        assert int(c.err.item()) == binding.GDN_DEVERR_TOKEN


def test_a_row_without_any_probability():
    c = Case(new=[1, 1], vocab=64, seed=11)
    c.p[0] = 0.0
    acc, nxt = c.run()
    assert acc.tolist() == [1, 1] and nxt[0] == -1 and nxt[1] >= 0
    assert int(c.err.item()) == binding.GDN_DEVERR_TOKEN


def test_bad_offsets_flag_and_skip():
    c = Case(new=[3, 2, 4, 1], vocab=50, seed=12)
    good = oracle.accept_sample(c.ids, c.p, c.q, c.u, c.us, c.cu)
    bad = torch.tensor([0, 3, 2, 9, 11], dtype=torch.int32, device="cuda")
    # request 1 has a negative length, 2 more than max_T, 3 runs past the rows
    acc, nxt = c.run(cu_seqlens=bad)
    assert int(c.err.item()) == binding.GDN_DEVERR_SEQLEN
    assert acc.tolist() == [good[0][0], -9, -9, -9] and nxt.tolist() == [good[1][0], -9, -9, -9]


def test_same_result_in_a_graph_and_on_another_stream():
    c = Case(new=[4, 6, 1, 3] * 10, vocab=30000, seed=13)
    c.check()
    acc, nxt = c.acc.clone(), c.nxt.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.gdn_accept_sample(c.sample, c.acc, c.nxt)
    c.acc.zero_()
    c.nxt.zero_()
    with torch.cuda.stream(s):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(acc, c.acc) and torch.equal(nxt, c.nxt)


def test_offsets_beyond_32_bits():
    # rows behind 2^31 elements: two requests of one row each, far apart in one allocation
    stride = (1 << 31) + 8
    flat = torch.zeros(stride + 1000, device="cuda")
    p = flat.as_strided((2, 1000), (stride, 1))
    c = Case(new=[1, 1], vocab=1000, seed=14, lookup=True)
    p.copy_(torch.from_numpy(c.p))
    c.check(target_probs=p)
