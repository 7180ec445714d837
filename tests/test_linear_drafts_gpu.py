"""Outputs of drafts (gdn_linear_verify) in bfloat16: the kernel for fewer than 48 rows at every count of 16-row groups,
blocks that take several units in turn, and the prompts' kernel with its longest requests first.

Tolerances are those of test_linear_gpu.py, and for fewer than 48 rows 2^-17 of each term besides: the state, and the
weights of the values, enter their products as two bfloat16 terms, of which the first is off by at most half
a step, 2^-8 of 1 to 2, and the second by half a step of that, 2^-17.

What is compared bit for bit (good requests among bad ones, a graph's replay) is the same sums in the same order."""
import numpy as np
import pytest
import torch

from speculative_decode_gated_gb300 import binding
from test_linear_gpu import TILES, Case

pytestmark = pytest.mark.gpu


class Drafts(Case):
    def tolerance(self, value, mag, state):
        tol = super().tolerance(value, mag, state)
        if not state and self.dtype == "bf16" and 1 < self.max_T < TILES:
            tol = tol + 2.0 ** -17 * (1 + 2.0 ** -8) * mag
        return tol


def verified(c, **over):
    o = c.output()
    binding.gdn_linear_verify(c.make(**over), o)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("heads,k_heads,dk,dv", [(2, 1, 64, 64), (3, 3, 64, 128), (2, 2, 128, 128), (6, 2, 128, 192),
                                                 (2, 2, 64, 256)])
@pytest.mark.parametrize("gates", ["token", "head", "none"])
@pytest.mark.parametrize("T", [2, 15, 16, 17, 32, 33, 47])
def test_rows(T, gates, heads, k_heads, dk, dv):
    c = Drafts(new=[T, 1, 0, T // 2 + 1, T], heads=heads, k_heads=k_heads, dk=dk, dv=dv, gates=gates, seed=T,
               sliced=True)
    c.check(verified(c))


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("T", [2, 16, 17, 47, 48, 200])
def test_uniform_rows(T, dk):
    c = Drafts(new=[T] * 3, heads=3, dk=dk, ragged=False, seed=100 + T)
    c.check(verified(c))


@pytest.mark.parametrize("T", [2, 12, 40, 140])
def test_a_decay_of_zero_forgets(T):
    c = Drafts(new=[T, T], heads=2, seed=61)
    cut = T // 2
    c.g[[cut, T + cut]] = -np.inf
    c.dg[[cut, T + cut]] = -float("inf")
    c.check(verified(c))


@pytest.mark.parametrize("T", [12, 40, 140])
def test_steep_decays(T):
    c = Drafts(new=[T, T], heads=2, seed=62, decay=40.0)
    c.check(verified(c))


# Units that are more than twice what runs at once (304 blocks), and no multiple of it: blocks take several in turn.
@pytest.mark.parametrize("B,heads,k_heads,dk,dv,T", [(50, 16, 8, 64, 64, 16), (21, 10, 5, 128, 192, 9),
                                                     (27, 12, 12, 128, 128, 47), (41, 16, 4, 64, 64, 33)])
def test_many_units(B, heads, k_heads, dk, dv, T):
    rng = np.random.default_rng(B)
    new = [int(x) for x in rng.integers(0, T + 1, B)]
    new[0], new[-1] = T, 0
    assert B * heads * dv // 64 > 2 * 304
    c = Drafts(new=new, heads=heads, k_heads=k_heads, dk=dk, dv=dv, seed=63)
    o = verified(c)
    c.check(o)
    # bad slots and offsets in the middle: these requests' rows stay, all others' keep every bit
    bad = sorted({1, B // 3, B // 2, B - 2})
    slots = c.dslots.clone()
    slots[bad] = torch.tensor([-1, B + 2, 2 ** 31 - 1, -2 ** 31][:len(bad)], dtype=torch.int32, device="cuda")
    again = verified(c, slot_ids=slots)
    assert int(c.err.item()) == binding.GDN_DEVERR_SLOT
    keep = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    for r in bad:
        keep[c.cu[r]:c.cu[r + 1]] = False
    assert torch.equal(again[keep], o[keep]) and bool((again[~keep] == 7).all())
    c.err.zero_()
    assert torch.equal(c.pool.cpu().view(torch.int32), c.pool0.view(torch.int32))


@pytest.mark.parametrize("T", [12, 40, 100])
def test_bad_offsets_are_skipped(T):
    c = Drafts(new=[T] * 5, seed=64)
    ref = verified(c)
    bad = c.dcu.clone()
    bad[2], bad[5] = T * 2 + T + 1, c.rows + 1      # request 1 too long, 2 short, 4 past the end
    o = verified(c, cu_seqlens=bad)
    assert int(c.err.item()) == binding.GDN_DEVERR_SEQLEN
    assert torch.equal(o[:T], ref[:T]) and torch.equal(o[3 * T:4 * T], ref[3 * T:4 * T])
    assert bool((o[T:2 * T] == 7).all()) and bool((o[4 * T:] == 7).all())


# More units than SMs and uneven prompts: blocks take the longest requests first.
@pytest.mark.parametrize("call", ["verify", "step", "commit"])
def test_prompts_longest_first(call):
    rng = np.random.default_rng(65)
    new = [int(x) for x in rng.integers(0, 150, 23)]
    new[3], new[7], new[8], new[22] = 300, 0, new[9], 129
    c = Drafts(new=new, heads=4, k_heads=2, dk=64, dv=128, seed=65)
    assert len(new) * 4 * 2 > 152
    if call == "commit":
        kept = [int(rng.integers(0, x + 1)) for x in new]
        binding.gdn_linear_commit(c.make(q=None), torch.tensor(kept, dtype=torch.int32, device="cuda"))
        c.check(rows=kept)
        return
    assert new[10] > 0 and 0 < new[11] + new[12] < 299
    o = c.output()
    (binding.gdn_linear_verify if call == "verify" else binding.gdn_linear_step)(c.lin, o)
    c.check(o, None if call == "verify" else new)
    if call == "verify":  # one request's offsets run backwards: it is skipped, and the next one begins a row early
        bad = c.dcu.clone()
        bad[12] = int(c.cu[11]) - 1
        again = verified(c, cu_seqlens=bad)
        assert int(c.err.item()) == binding.GDN_DEVERR_SEQLEN
        keep = torch.ones(c.rows, dtype=torch.bool, device="cuda")
        keep[c.cu[11] - 1:c.cu[13]] = False  # (the first of these is two requests', in either order)
        assert torch.equal(again[keep], o[keep])


@pytest.mark.parametrize("T", [2, 16, 40, 200])
def test_graph_replay_and_streams(T):
    # captured verifies of two problems on two streams, replayed at the same time, give the eager results
    cases = [Drafts(new=[T, max(1, T // 2)], seed=s, max_T=T) for s in (66, 67)]
    refs = [verified(c) for c in cases]
    outs = [c.output() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c, o, s in zip(cases, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            binding.gdn_linear_verify(c.lin, o)
        graphs.append(g)
    for _ in range(2):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, ref in zip(outs, refs):
            assert torch.equal(o, ref)


@pytest.mark.parametrize("T", [16, 40, 1000])
def test_the_same_bits_each_time(T):
    c = Drafts(new=[T, T // 3, T], heads=8, seed=68, gates="head")
    first = verified(c)
    other = Drafts(new=[50, 60], seed=69)
    for _ in range(4):
        verified(other)
        assert torch.equal(verified(c), first)
    states = []
    for _ in range(3):
        c.pool.copy_(c.pool0)
        binding.gdn_linear_step(c.lin, c.output())
        states.append(c.pool.clone())
    assert all(torch.equal(x.view(torch.int32), states[0].view(torch.int32)) for x in states)
