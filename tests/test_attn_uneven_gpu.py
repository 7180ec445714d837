"""GPU: drafts of one request with a long context among many with short ones.  The long
request's units lie in most of the workers; their partials must not be joined by one warpgroup.
Values against the oracle, and the time of the call against those of its two parts."""
import pytest
import torch

from attn_cases import Case, to_dev
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


def time_of(c):
    """Least time of a call over some replays of a graph of five."""
    q = to_dev(c.q, c.dtype)
    o = torch.empty_like(q)
    ws = binding.paged_attn_workspace(c.attn)
    binding.gdn_paged_attn(c.attn, q, o, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(5):
            binding.gdn_paged_attn(c.attn, q, o, workspace=ws)
    best = float("inf")
    for _ in range(20):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / 5)
    return best


@pytest.mark.parametrize("hd,T,G", [(128, 16, 8), (64, 16, 8), (128, 40, 8)])
def test_a_long_request_costs_what_it_costs_alone(hd, T, G):
    short = [17 * r % 90 for r in range(39)]

    def case(old):
        return Case(new=[T] * len(old), old=old, q_heads=2 * G, kv_heads=2, hd=hd, page=64,
                    seed=hd + T).device()

    together = case(short[:13] + [60000] + short[13:])
    # twice both calls one after the other; a warpgroup alone took some 1 us for each of 150 partials
    assert time_of(together) <= 2 * (time_of(case([60000])) + time_of(case(short)))


@pytest.mark.parametrize("hd,T,G", [(128, 16, 8), (64, 16, 8), (128, 40, 8), (64, 30, 8), (128, 24, 3)])
@pytest.mark.parametrize("long", [700, 9000])
def test_groups_of_partials(hd, T, G, long):
    # units of two or three partials, of one group and of several levels, next to each other
    # on the line
    old, new = [17 * r % 90 for r in range(60)], [r % 3 for r in range(60)]
    old[7], old[8], old[33] = long, long // 2, long // 5
    new[7], new[8], new[33] = T, T // 2, T
    c = Case(new=new, old=old, q_heads=2 * G, kv_heads=2, hd=hd, page=32, seed=hd + T + long).device()
    c.run().check()
    o, ws = c.o.clone(), c.ws
    assert not ws[9728:16384].any()              # the counters are back at zero
    assert torch.equal(c.run(workspace=ws).o, o)  # and the results the same from call to call
