"""Linear attention with a decay for each head (gdn_linear_verify, _commit, _step) against the
float64 oracle.

Tolerances.  Every term of an output or a state is a product of float32 factors: n decays, each off by
2^-22 of itself (its exponent's rounding within expf's error bound of 2 units in the last place), and
at most 8 further roundings; a sum of dk + n such terms in float32 adds at most 2^-24 a term.  With
n rows that is (4 n + dk + n + 8) 2^-24 of the sum of the terms' absolute values (`mag` of the oracle).
A bfloat16 output is rounded once: 2^-8 of itself.  In the prompts' kernel (bfloat16, max_T from 48 on)
states and weights are rounded to bfloat16 for o, 2^-8 of each term, and to two bfloat16 terms for what
is added to a state, 2^-16 of each term; a block's decays come from sums of up to 128 logarithms in two
float32 words, which lose less than the products above."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TILES = 48  # rows from which the prompts' kernel runs (bf16, dk 64 or 128, dv a multiple of 64)


def rounded(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return t.to(TYPES[dtype]).float().numpy()


class Case:
    """Requests with `new` rows each, in a pool whose other slots, and in arrays whose other rows, hold
    NaN.  Rows are slices of one wider array when `sliced`."""

    def __init__(self, *, new, heads=2, k_heads=None, dk=128, dv=128, dtype="bf16", gates="token", seed=0,
                 ragged=True, sliced=False, scale=0.7, max_T=None, extra=3, decay=1.0):
        rng = np.random.default_rng(seed)
        self.new, self.H, self.dk, self.dv, self.dtype, self.scale = list(new), heads, dk, dv, dtype, scale
        self.Hk = heads if k_heads is None else k_heads
        self.B, n = len(new), sum(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.rows, self.n = n + (extra if ragged else 0), n
        self.max_T = max(list(new) + [0]) if max_T is None else max_T
        self.q = rounded(rng.standard_normal((n, self.Hk, dk)), dtype)
        self.k = rounded(rng.standard_normal((n, self.Hk, dk)) * dk ** -0.5, dtype)
        self.v = rounded(rng.standard_normal((n, heads, dv)), dtype)
        self.g = (-rng.random((n, heads) if gates == "token" else heads) * 0.3 * decay).astype(np.float32)
        if gates == "none":
            self.g = np.zeros(heads, np.float32)
        self.s0 = rng.standard_normal((self.B, heads, dk, dv)).astype(np.float32)
        self.slots = rng.permutation(self.B + 2)[:self.B].astype(np.int32)
        self.pool0 = torch.full((self.B + 2, heads, dk, dv), float("nan"))
        self.pool0[self.slots.astype(np.int64)] = torch.from_numpy(self.s0)

        def device(x, cols):
            y = torch.full((self.rows, cols + (32 if sliced else 0)) + x.shape[2:], float("nan"),
                           dtype=TYPES[dtype], device="cuda")
            y[:n, :cols] = torch.from_numpy(x).to(TYPES[dtype]).cuda()
            return y[:, :cols]

        self.dq, self.dk_, self.dv_ = device(self.q, self.Hk), device(self.k, self.Hk), device(self.v, heads)
        self.dg = torch.from_numpy(self.g).cuda()
        if self.g.ndim == 2:
            self.dg = torch.full((self.rows, heads), float("nan"), device="cuda")
            self.dg[:n] = torch.from_numpy(self.g).cuda()
        self.pool = self.pool0.cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.dcu = torch.from_numpy(self.cu.astype(np.int32)).cuda() if ragged else None
        self.dslots = torch.from_numpy(self.slots).cuda()
        self.lin = self.make()

    def make(self, **over):
        kw = dict(q=self.dq, k=self.dk_, v=self.dv_, log_decay=self.dg, pool=self.pool,
                  slot_ids=self.dslots, max_T=self.max_T, cu_seqlens=self.dcu, scale=self.scale,
                  dev_err=self.err)
        kw.update(over)
        return binding.make_linear(**kw)

    def output(self):
        return torch.full((self.rows, self.H, self.dv), 7.0, dtype=TYPES[self.dtype], device="cuda")

    def tolerance(self, value, mag, state):
        n = max(self.new + [1])
        tol = (5 * n + self.dk + 8) * 2.0 ** -24 * mag
        tiles = (self.dtype == "bf16" and self.max_T >= TILES and self.dk in (64, 128)
                 and self.dv % 64 == 0)
        if state:
            return tol + (2.0 ** -16 * mag if tiles else 0) + 1e-30
        if self.dtype == "bf16":
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(value)
        return tol + (2.0 ** -8 * (1 + 2.0 ** -8) * mag if tiles else 0) + 1e-30

    def check(self, o=None, rows=None, states=True):
        """rows: of each request, those in its state afterwards (None: the states stay)."""
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        if o is not None:
            want, _, mag, _ = oracle.linear_attention(self.q, self.k, self.v, self.g, self.s0, self.cu, self.scale)
            got = o.float().cpu().numpy()
            assert np.all(got[self.n:] == 7.0)  # rows that no request has
            off = np.abs(got[:self.n] - want)
            tol = self.tolerance(want, mag, False)
            assert np.all(off <= tol), float(np.max(off / tol))
        pool = self.pool.cpu()
        if rows is None:
            assert torch.equal(pool.view(torch.int32), self.pool0.view(torch.int32))
            return
        _, want, _, mag = oracle.linear_attention(self.q, self.k, self.v, self.g, self.s0, self.cu, self.scale,
                                                  rows)
        got = pool.numpy()
        for r, slot in enumerate(self.slots):
            if rows[r] == 0:
                assert np.array_equal(got[slot], self.s0[r])
        off = np.abs(got[self.slots] - want)
        tol = self.tolerance(want, mag, True)
        assert np.all(off <= tol), float(np.max(off / tol))
        others = np.setdiff1d(np.arange(self.B + 2), self.slots)
        assert np.all(np.isnan(got[others]))


SHAPES = [  # heads, k_heads, dk, dv
    (1, 1, 32, 32), (3, 1, 32, 64), (2, 2, 64, 64), (4, 2, 64, 96), (2, 2, 64, 256), (2, 1, 128, 32),
    (3, 3, 128, 64), (2, 2, 128, 128), (6, 2, 128, 192), (2, 2, 256, 128), (2, 1, 256, 32),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,k_heads,dk,dv", SHAPES)
@pytest.mark.parametrize("new", [[1], [1, 1, 0, 1], [2, 17, 0, 16, 33, 1]])
def test_step(new, heads, k_heads, dk, dv, dtype):
    c = Case(new=new, heads=heads, k_heads=k_heads, dk=dk, dv=dv, dtype=dtype)
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,k_heads,dk,dv", SHAPES)
def test_verify_then_commit(heads, k_heads, dk, dv, dtype):
    c = Case(new=[5, 16, 0, 3, 21], heads=heads, k_heads=k_heads, dk=dk, dv=dv, dtype=dtype, gates="head",
             sliced=True, seed=1)
    o = c.output()
    binding.gdn_linear_verify(c.lin, o)
    c.check(o)
    kept = [5, 0, 0, 1, 18]
    acc = torch.tensor(kept, dtype=torch.int32, device="cuda")
    binding.gdn_linear_commit(c.make(q=None), acc)
    c.check(rows=kept)


# Rows of the prompts' kernel: whole blocks of 128, one more, one fewer, many blocks.
@pytest.mark.parametrize("heads,k_heads,dk,dv", [(2, 1, 64, 64), (2, 2, 128, 128), (3, 3, 128, 64), (2, 2, 64, 256),
                                                 (4, 2, 128, 192), (2, 2, 256, 128), (2, 2, 128, 96)])
@pytest.mark.parametrize("new", [[48], [128, 0, 127, 129, 1], [300, 513]])
def test_prompts(new, heads, k_heads, dk, dv):
    c = Case(new=new, heads=heads, k_heads=k_heads, dk=dk, dv=dv, sliced=True, seed=2)
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


@pytest.mark.parametrize("gates,decay", [("head", 1.0), ("none", 1.0), ("token", 30.0)])
def test_prompt_decays(gates, decay):
    c = Case(new=[200, 70], gates=gates, decay=decay, seed=3)
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


def test_prompt_verify_and_commit():
    c = Case(new=[150, 64, 260], seed=4)
    o = c.output()
    binding.gdn_linear_verify(c.lin, o)
    c.check(o)
    kept = [131, 0, 128]
    binding.gdn_linear_commit(c.lin, torch.tensor(kept, dtype=torch.int32, device="cuda"))
    c.check(rows=kept)


@pytest.mark.parametrize("T", [1, 7, 16, 130])
def test_uniform_rows(T):
    c = Case(new=[T] * 5, heads=3, ragged=False, seed=5)
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


@pytest.mark.parametrize("T", [1, 9, 140])
def test_a_decay_of_zero_forgets(T):
    # from the row with g = -infinity on, nothing of the rows and the state before is left
    c = Case(new=[T, T], heads=2, seed=6)
    cut = T // 2
    c.g[[cut, T + cut]] = -np.inf
    c.dg[[cut, T + cut]] = -float("inf")
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    c.check(o, c.new)


def test_grouped_heads_and_stride_of_the_decays():
    c = Case(new=[20, 90], heads=8, k_heads=2, dk=64, dv=64, seed=7)
    wide = torch.full((c.rows, 8 + 5), float("nan"), device="cuda")
    wide[:, :8] = c.dg
    o = c.output()
    binding.gdn_linear_step(c.make(log_decay=wide[:, :8]), o)
    c.check(o, c.new)


@pytest.mark.parametrize("T", [1, 12, 100])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_aligned_to_16_bytes_only(T, dtype):
    c = Case(new=[T, T + 1], heads=2, seed=14, dtype=dtype)
    step = 16 // (2 if dtype == "bf16" else 4)

    def moved(x):  # a row 16 bytes longer than its heads, from 16 bytes behind an allocation's start
        n, h, d = x.shape
        flat = torch.full((n * (h * d + step) + step,), float("nan"), dtype=x.dtype, device="cuda")
        y = flat[step:].view(n, h * d + step)[:, :h * d].view(n, h, d)
        y.copy_(x)
        return y

    o = torch.full((c.rows * 2 * 128 + step,), 7.0, dtype=TYPES[dtype], device="cuda")[step:].view(c.rows, 2, 128)
    binding.gdn_linear_step(c.make(q=moved(c.dq), k=moved(c.dk_), v=moved(c.dv_)), o)
    c.check(o, c.new)


@pytest.mark.parametrize("T", [1, 12, 100])
def test_bad_requests_are_skipped(T):
    c = Case(new=[T] * 5, seed=8)
    bad = c.dcu.clone()
    bad[2], bad[5] = T * 2 + T + 1, c.rows + 1      # request 1 too long, 2 short, 4 past the end
    slots = c.dslots.clone()
    slots[0] = c.pool.shape[0]
    o = c.output()
    binding.gdn_linear_step(c.make(cu_seqlens=bad, slot_ids=slots), o)
    torch.cuda.synchronize()
    assert int(c.err.item()) == binding.GDN_DEVERR_SEQLEN | binding.GDN_DEVERR_SLOT
    assert bool((o[:T] == 7).all()) and bool((o[4 * T:] == 7).all())
    pool = c.pool.cpu()
    for r in (0, 1, 4):
        assert torch.equal(pool[c.slots[r]].view(torch.int32), c.pool0[c.slots[r]].view(torch.int32))
    good = Case(new=[T] * 5, seed=8)
    binding.gdn_linear_step(good.lin, good.output())
    assert torch.equal(pool[c.slots[3]], good.pool[c.slots[3]].cpu())
    c.err.zero_()
    kept = torch.tensor([T, -1, T + 1, 0, T], dtype=torch.int32, device="cuda")
    before = c.pool.clone()
    binding.gdn_linear_commit(c.lin, kept)
    assert int(c.err.item()) == binding.GDN_DEVERR_ACCEPTED
    for r in (1, 2, 3):
        assert torch.equal(c.pool[c.slots[r]].view(torch.int32), before[c.slots[r]].view(torch.int32))


@pytest.mark.parametrize("T", [1, 12, 100])
def test_values_that_are_not_finite_stay_with_their_head(T):
    c = Case(new=[T, T, T], heads=2, seed=9)
    c.dv_[T + T // 2, 0, 3] = float("inf")
    c.dk_[2 * T + T // 2, 1, 5] = float("nan")
    ref = Case(new=[T, T, T], heads=2, seed=9)
    o, o_ref = c.output(), ref.output()
    binding.gdn_linear_step(c.lin, o)
    binding.gdn_linear_step(ref.lin, o_ref)
    same = torch.ones_like(o, dtype=torch.bool)
    start = 0 if T >= TILES else T // 2
    same[T + start:2 * T, 0] = False
    same[2 * T + start:3 * T, 1] = False
    assert torch.equal(o[same], o_ref[same])
    assert not bool(torch.isfinite(c.pool[c.slots[1], 0, :, 3]).all())
    assert bool(torch.isnan(c.pool[c.slots[2], 1, 5]).all())
    assert torch.equal(c.pool[c.slots[0]], ref.pool[c.slots[0]])
    assert torch.equal(c.pool[c.slots[1], 1], ref.pool[c.slots[1], 1])


@pytest.mark.parametrize("T", [1, 16, 200])
def test_graph_replay_and_streams(T):
    # two captured graphs on two streams, replayed at the same time, give the eager results
    cases = [Case(new=[T, max(1, T // 2)], seed=s, max_T=T) for s in (10, 11)]
    eager = [Case(new=[T, max(1, T // 2)], seed=s, max_T=T) for s in (10, 11)]
    outs, refs = [c.output() for c in cases], [c.output() for c in eager]
    for _ in range(2):
        for c, o in zip(eager, refs):
            binding.gdn_linear_step(c.lin, o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c, o, s in zip(cases, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.gdn_linear_step(c.lin, o)
        graphs.append(g)
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, e, o, ref in zip(cases, eager, outs, refs):
        assert torch.equal(o, ref)
        assert torch.equal(c.pool.view(torch.int32), e.pool.view(torch.int32))


def test_a_prompt_and_its_rows_one_by_one():
    # the same rows in one call and in single-row calls, float32: (the tolerance, twice)
    c = Case(new=[40, 40], dtype="fp32", gates="head", seed=12, ragged=False)
    one = Case(new=[40, 40], dtype="fp32", gates="head", seed=12, ragged=False)
    o, rows = c.output(), one.output()
    binding.gdn_linear_step(c.lin, o)
    for t in range(40):
        at = torch.tensor([t, 40 + t], device="cuda")
        part = torch.empty((2, 2, 128), device="cuda")
        binding.gdn_linear_step(binding.make_linear(
            q=one.dq[at], k=one.dk_[at], v=one.dv_[at], log_decay=one.dg, pool=one.pool,
            slot_ids=one.dslots, max_T=1, scale=one.scale), part)
        rows[at] = part
    c.check(o, c.new)
    one.check(rows, c.new)


def test_no_requests_and_no_rows():
    c = Case(new=[0, 0], max_T=4)
    binding.gdn_linear_step(c.lin, c.output())
    binding.gdn_linear_commit(c.lin, torch.zeros(2, dtype=torch.int32, device="cuda"))
    c.check(rows=[0, 0])


def test_more_units_than_any_launch_dimension_but_the_first():
    c = Case(new=[1] * 300, heads=230, dk=32, dv=32, seed=13, ragged=False)  # 69000 units
    o = c.output()
    binding.gdn_linear_step(c.lin, o)
    torch.cuda.synchronize()
    k, v, g = c.dk_.float(), c.dv_.float(), c.dg
    s = c.pool0.cuda()[c.dslots.long()] * g.exp()[..., None, None] + k[..., :, None] * v[..., None, :]
    want = (c.dq.float()[..., None, :] @ s)[..., 0, :] * c.scale
    assert float((o.float() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) * 1.01
    assert float((c.pool[c.dslots.long()] - s).abs().max()) <= 2.0 ** -20 * float(s.abs().max())
