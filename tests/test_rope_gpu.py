"""GPU parity of rotary positions with the append to the pages against the float64
oracle: both pair layouts, parts of the head, scaled frequencies, far positions, ragged
rows, and which places of the cache are written.

Tolerance: cosine and sine are float32 with an absolute error below 2^-21 (the angle's
fraction of a turn is rounded to 2^-25), so an element is off by at most
2^-20 (|x| + |y|) mscale, and a bf16 result by half a unit of its 8-bit significand more."""
import numpy as np
import pytest
import torch

import oracle
from attn_cases import TYPES, rounded, to_dev
from speculative_decode_gated_gb300 import binding, staging

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, *, new, old, q_heads=4, kv_heads=2, hd=64, page=16, dtype="bf16", rot=None,
                 interleaved=False, seed=0, positions=None, ragged=True, **freq):
        rng = np.random.default_rng(seed)
        rot = hd if rot is None else rot
        self.new, self.old, self.dtype, self.page, self.hd = new, old, dtype, page, hd
        self.q_heads, self.kv_heads, self.interleaved = q_heads, kv_heads, interleaved
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        n = int(self.cu[-1])
        span = [(o // page, (o + t + page - 1) // page) for o, t in zip(old, new)]
        self.width = max(b for _, b in span) + 1
        n_pages = sum(b - a for a, b in span) + 2
        ids, at = rng.permutation(n_pages), 0
        self.table = np.full((len(new), self.width), -3, np.int32)
        for r, (a, b) in enumerate(span):
            self.table[r, a:b] = ids[at:at + b - a]
            at += b - a
        self.pages0 = rounded(rng.standard_normal((2, n_pages, kv_heads, page, hd)), dtype)
        rows = rounded(rng.standard_normal((n, q_heads + 2 * kv_heads, hd)), dtype)
        self.rows = rows
        self.q, self.k = rows[:, :q_heads], rows[:, q_heads:q_heads + kv_heads]
        self.v = rows[:, q_heads + kv_heads:]
        f, self.mscale = staging.rope_frequencies(rot, device="cuda", **freq)
        self.f = f.cpu().numpy().astype(np.float64)
        place = np.concatenate([o + np.arange(t) for o, t in zip(old, new)])
        self.pos = place if positions is None else np.asarray(positions)
        d = to_dev(rows, dtype)
        self.dq, self.dk = d[:, :q_heads], d[:, q_heads:q_heads + kv_heads]
        self.dv = d[:, q_heads + kv_heads:]
        self.dkp, self.dvp = to_dev(self.pages0[0], dtype), to_dev(self.pages0[1], dtype)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlen = torch.tensor(old, dtype=torch.int32, device="cuda")
        self.dcu = torch.from_numpy(self.cu).cuda() if ragged else None
        self.attn = binding.make_attn(q_heads=q_heads, k_pages=self.dkp, v_pages=self.dvp,
                                      page_table=self.dtable, kv_len=self.dlen, max_T=max(new),
                                      cu_seqlens=self.dcu, n_tok=n, dev_err=self.err)
        self.rope = binding.make_rope(
            inv_freq=f, interleaved=interleaved, mscale=self.mscale,
            positions=None if positions is None else torch.tensor(self.pos, dtype=torch.int32,
                                                                  device="cuda"))
        self.out = torch.full((n, q_heads, hd), 7.0, dtype=TYPES[dtype], device="cuda")

    def run(self, stream=None):
        binding.gdn_rope_append(self.attn, self.rope, self.dq, self.dk, self.dv, self.out, stream)
        torch.cuda.synchronize()
        return self

    def near(self, got, want, x):
        """x: the values before the turn, for the tolerance (a pair's sum bounds both)."""
        both = np.abs(x) + np.max(np.abs(x), axis=-1, keepdims=True)
        tol = 2.0 ** -20 * both * self.mscale
        if self.dtype == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))

    def check(self, rows=None):
        rows = np.arange(self.cu[-1]) if rows is None else np.asarray(rows)
        turn = lambda x: oracle.rope(x, self.pos, self.f, self.interleaved, self.mscale)  # noqa: E731
        self.near(self.out.float().cpu().numpy()[rows], turn(self.q)[rows], self.q[rows])
        kt = turn(self.k)
        want = [self.pages0[0].astype(np.float64), self.pages0[1].astype(np.float64)]
        plain = self.pages0[0].astype(np.float64)
        for r in range(len(self.new)):
            here = slice(self.cu[r], self.cu[r + 1])
            if self.cu[r] in rows:
                oracle.write_rows(want[0], self.table, r, self.old[r], kt[here])
                oracle.write_rows(want[1], self.table, r, self.old[r], self.v[here])
                oracle.write_rows(plain, self.table, r, self.old[r], self.k[here])
        assert np.array_equal(self.dvp.float().cpu().numpy(), want[1])  # values are moved, not rounded
        got = self.dkp.float().cpu().numpy()
        same = want[0] == self.pages0[0]  # places that nothing writes keep their bits
        assert np.array_equal(got[same & (plain == self.pages0[0])],
                              self.pages0[0][same & (plain == self.pages0[0])])
        self.near(got, want[0], plain)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hd,rot", [(32, 32), (32, 16), (64, 64), (64, 48), (128, 128), (128, 32),
                                    (256, 256), (256, 64), (128, 112)])
def test_heads_and_parts(dtype, interleaved, hd, rot):
    Step(new=[3, 1, 0, 17], old=[5, 15, 4, 300], hd=hd, rot=rot, dtype=dtype,
         interleaved=interleaved, seed=hd + rot).run().check()


@pytest.mark.parametrize("heads", [(1, 1), (5, 5), (32, 8), (64, 1), (15, 3)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_head_counts_and_pages(heads, page):
    Step(new=[40, 2], old=[page - 1, 3 * page], q_heads=heads[0], kv_heads=heads[1], hd=128,
         page=page, seed=page).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 8.0),
                                            ("yarn", 32.0)])
@pytest.mark.parametrize("old", [0, 4095, 131071, 16777213])
def test_far_positions(dtype, scaling, factor, old):
    # beyond 2^24 a float32 cannot hold the position itself
    Step(new=[6], old=[old], dtype=dtype, page=256, scaling=scaling, factor=factor, base=500000.0,
         seed=old % 97).run().check()


@pytest.mark.parametrize("interleaved", [False, True])
def test_given_positions(interleaved):
    Step(new=[4, 3], old=[9, 2], positions=[0, 0, 7, -5, 1 << 30, 100, 3], interleaved=interleaved,
         dtype="fp32", seed=4).run().check()


def test_uniform_rows():
    Step(new=[16] * 5, old=[1, 2, 3, 100, 17], ragged=False, hd=128, seed=8).run().check()


def test_values_pass_unchanged_whatever_they_are():
    s = Step(new=[2], old=[3], seed=1)
    s.dv[0, 0, :3] = torch.tensor([float("nan"), float("inf"), -0.0])
    s.run()
    page = s.dvp[int(s.table[0, 0]), 0, 3].view(torch.int16)
    assert torch.equal(page, s.dv[0, 0].contiguous().view(torch.int16))


def test_bad_requests_and_pages():
    s = Step(new=[2, 3, 4, 2], old=[3, 20, 9, 30], seed=2)
    s.dlen[1] = -2
    s.dlen[3] = s.width * s.page - 1
    s.run()
    assert int(s.err.item()) == binding.GDN_DEVERR_KV_LEN
    assert torch.all(s.out[2:5] == 7) and torch.all(s.out[9:] == 7)
    s.check(rows=[0, 1, 5, 6, 7, 8])

    s = Step(new=[2, 3], old=[3, 20], seed=3)
    s.dtable[1, 1] = 10 ** 6
    s.run()
    assert int(s.err.item()) == binding.GDN_DEVERR_PAGE
    want = oracle.rope(s.q, s.pos, s.f)
    s.near(s.out.float().cpu().numpy(), want, s.q)     # every query is rotated
    s.table[1, 1] = s.table[0, 0]
    got = s.dvp.float().cpu().numpy()
    want = s.pages0[1].astype(np.float64)
    oracle.write_rows(want, s.table, 0, 3, s.v[:2])
    assert np.array_equal(got, want)                   # and nothing of request 1 is written

    s = Step(new=[2, 3, 0], old=[3, 20, 1], seed=3)
    s.dcu[3] = 99
    s.run()
    assert int(s.err.item()) == binding.GDN_DEVERR_SEQLEN
    s.check()


def test_pages_beyond_2_32_elements():
    s = Step(new=[3, 2], old=[14, 40], hd=128, seed=6).run()
    n = (1 << 32) // (2 * 16 * 128) + 9
    big = [torch.zeros((n,) + s.dkp.shape[1:], dtype=s.dkp.dtype, device="cuda") for _ in range(2)]
    m = s.dkp.shape[0]
    for b, p in zip(big, s.pages0):
        b[n - m:] = to_dev(p, "bf16")
    table = torch.where(s.dtable >= 0, s.dtable + (n - m), s.dtable)
    attn = binding.make_attn(q_heads=4, k_pages=big[0], v_pages=big[1], page_table=table,
                             kv_len=s.dlen, max_T=3, cu_seqlens=s.dcu, n_tok=5, dev_err=s.err)
    binding.gdn_rope_append(attn, s.rope, s.dq, s.dk, s.dv, s.out)
    torch.cuda.synchronize()
    assert torch.equal(big[0][n - m:], s.dkp) and torch.equal(big[1][n - m:], s.dvp)
    assert int(s.err.item()) == 0


def test_streams_and_graphs():
    s = Step(new=[16] * 4, old=[1, 22, 300, 64], hd=128, ragged=False, seed=5).run()
    want = s.out.clone(), s.dkp.clone(), s.dvp.clone()
    for t, p in ((s.dkp, s.pages0[0]), (s.dvp, s.pages0[1])):
        t.copy_(to_dev(p, "bf16"))
    s.out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.gdn_rope_append(s.attn, s.rope, s.dq, s.dk, s.dv, s.out)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (s.out, s.dkp, s.dvp)):
        assert torch.equal(a, b)
    s.out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.run(side)
    assert torch.equal(s.out, want[0])
