"""The next step's pages (gdn_plan_pages) against the oracle: every number has to be equal."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decode_gated_gb300 import binding

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Cache:
    """A paged cache's bookkeeping on the device, in place, beside the oracle's lists."""

    def __init__(self, batch, page, width, n_pages, max_T, seed=0, slots=True, positions=True, max_rows=None):
        rng = np.random.default_rng(seed)
        self.B, self.page, self.width, self.n_pages, self.max_T = batch, page, width, n_pages, max_T
        self.kv_len, self.held = [0] * batch, [0] * batch
        self.table = [[-1] * width for _ in range(batch)]
        self.free = [int(x) for x in rng.permutation(n_pages)]
        self.d = dict(kv_len=i32(self.kv_len), held=i32(self.held), page_table=i32(self.table).reshape(batch, width),
                      free_pages=i32(self.free), free_count=i32([n_pages]), cu_seqlens=i32([-1] * (batch + 1)))
        size = batch * max_T if max_rows is None else max_rows
        self.slots = torch.empty(size, dtype=torch.int64, device="cuda") if slots else None
        self.positions = torch.empty(size, dtype=torch.int32, device="cuda") if positions else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def plan(self, rows=None, accepted=None, done=None, page_size=None, **over):
        for t in (self.slots, self.positions):
            if t is not None:
                t.fill_(-3)
        self.err.zero_()
        p = binding.make_pages(**{**self.d, **dict(
            page_size=self.page, max_T=self.max_T, rows=None if rows is None else i32(rows),
            accepted=None if accepted is None else i32(accepted), done=None if done is None else i32(done),
            slots=self.slots, positions=self.positions, dev_err=self.err), **over})
        binding.gdn_plan_pages(p)
        torch.cuda.synchronize()
        return p

    def want(self, rows=None, accepted=None, done=None):
        return oracle.plan_pages(self.kv_len, self.held, self.free, self.table, self.page, self.max_T,
                                 self.n_pages, rows, accepted, done)

    def compare(self, w, kv_len=None, held=None, count=None, err=None):
        d = self.d
        assert (d["kv_len"] if kv_len is None else kv_len).tolist() == [int(x) for x in w["kv_len"]]
        assert (d["held"] if held is None else held).tolist() == [int(x) for x in w["held"]]
        n = len(w["free"])
        assert int((d["free_count"] if count is None else count).item()) == n
        assert d["free_pages"][:n].tolist() == [int(x) for x in w["free"]]
        table = d["page_table"].cpu().numpy()
        for r in range(self.B):
            assert table[r, :w["held"][r]].tolist() == [int(x) for x in w["table"][r][:w["held"][r]]]
        assert d["cu_seqlens"].tolist() == w["cu"]
        for t, name in ((self.slots, "slots"), (self.positions, "positions")):
            if t is not None:
                m = min(w["cu"][-1], t.numel())
                assert t[:m].tolist() == [int(x) for x in w[name][:m]]
                assert bool((t[m:] == -3).all())  # what lies behind the last row is left
        assert int(self.err.item()) == (w["err"] if err is None else err)

    def move_on(self, w):
        self.kv_len, self.held, self.free, self.table = w["kv_len"], w["held"], w["free"], w["table"]

    def step(self, rows=None, accepted=None, done=None):
        w = self.want(rows, accepted, done)
        self.plan(rows, accepted, done)
        self.compare(w)
        self.move_on(w)
        return w


@pytest.mark.parametrize("batch,page,max_T,n_pages,width", [
    (1, 16, 1, 30, 20), (1, 16, 300, 200, 60), (5, 16, 16, 60, 30), (33, 32, 40, 300, 25),
    (64, 16, 16, 900, 40), (200, 64, 100, 700, 12), (1000, 16, 50, 6000, 20),
    (1024, 16, 8, 3000, 10), (1025, 16, 8, 3000, 10), (3000, 16, 5, 9000, 8), (40, 256, 3000, 400, 20),
])
def test_steps_of_a_cache(batch, page, max_T, n_pages, width):
    rng = np.random.default_rng(batch)
    c = Cache(batch, page, width, n_pages, max_T, seed=batch)
    rows = [0] * batch
    refused = 0
    for step in range(8):
        accepted = [int(rng.integers(0, t + 1)) for t in rows]
        wanted = [int(rng.integers(0, max_T + 1)) for _ in range(batch)]
        done = [int(c.kv_len[r] + accepted[r] + wanted[r] > width * page or rng.random() < 0.08)
                for r in range(batch)]
        w = c.step(wanted, accepted if step else None, done)
        rows = [b - a for a, b in zip(w["cu"], w["cu"][1:])]
        refused += w["err"] != 0
        used = [x for r in range(batch) for x in w["table"][r][:w["held"][r]]]
        assert sorted(used + w["free"]) == list(range(n_pages))


@pytest.mark.parametrize("slots,positions", [(False, False), (True, False), (False, True)])
def test_without_slots_or_positions(slots, positions):
    c = Cache(70, 16, 10, 600, 20, slots=slots, positions=positions)
    c.step()
    c.step(accepted=[r % 21 for r in range(70)])


def test_too_few_pages_go_to_the_first_requests():
    c = Cache(6, 16, 8, 10, 48)
    w = c.step(rows=[48, 48, 16, 48, 10, 0])   # 3 + 3 + 1 pages, then 3 of 3, then none
    assert w["cu"] == [0, 48, 96, 112, 160, 160, 160] and w["err"] == 256
    # one that wants none goes on; lengths move in any case
    w = c.step(rows=[0, 48, 48, 0, 16, 0], accepted=[48, 17, 16, 48, 0, 0])
    assert w["err"] == 256 and w["kv_len"] == [48, 17, 16, 48, 0, 0]
    # an ended request gives its 3 pages to those that come before it too: request 0 takes 2 (for 78
    # places, of which it holds 48), 1 has enough, 2 wants 3 more and 4 wants 1, both in vain
    w = c.step(rows=[30, 30, 48, 0, 16, 0], done=[0, 0, 0, 1, 0, 0])
    assert w["err"] == 256 and w["held"] == [5, 3, 1, 0, 0, 0] and len(w["free"]) == 1


def test_in_place_and_apart_are_the_same():
    apart = Cache(50, 16, 12, 400, 30, seed=1)
    for c in (apart,):
        c.step()
    kept = [r % 31 for r in range(50)]
    w = apart.want(None, kept)
    out = dict(kv_len_out=i32([9] * 50), held_out=i32([9] * 50), free_count_out=i32([9]))
    before = {k: apart.d[k].clone() for k in ("kv_len", "held", "free_count")}
    for _ in range(2):  # planned twice from the same lengths: the same step
        apart.plan(None, kept, **out)
        apart.compare(w, out["kv_len_out"], out["held_out"], out["free_count_out"])
        for k, x in before.items():
            assert torch.equal(apart.d[k], x)
        # (the list's end was taken, and stays where it is)


def test_bad_requests_stay_as_they_are():
    c = Cache(8, 16, 4, 60, 16)
    c.step()
    cases = [  # rows, accepted, kv_len, held of request 3 -> bit
        (17, 0, 0, 1, 4), (-1, 0, 0, 1, 4), (4, -1, 0, 1, 2), (4, 17, 0, 1, 2), (4, 0, -2, 1, 32),
        (4, 0, 0, 5, 32), (4, 0, 0, -1, 32),
    ]
    for rows, acc, kv, held, bit in cases:
        d = Cache(8, 16, 4, 60, 16)
        d.step()
        d.kv_len[3], d.held[3] = kv, held
        d.d["kv_len"][3], d.d["held"][3] = kv, held
        r, a = [8] * 8, [5] * 8
        r[3], a[3] = rows, acc
        w = d.want(r, a)
        assert w["err"] == bit
        d.plan(r, a)
        d.held[3] = w["held"][3] = max(0, min(held, 4)) if held != 5 else 4
        got_held = d.d["held"].clone()
        got_held[3] = d.held[3]  # (a number that is no count of pages is left as it was)
        assert int(d.d["held"][3].item()) == held
        d.compare(w, held=got_held)


def test_longer_than_the_table():
    c = Cache(3, 16, 3, 40, 30)
    c.step()
    w = c.step(rows=[30, 18, 19], accepted=[30, 30, 30])  # places 60, 48 and 49 of 48
    assert w["err"] == 32 and w["cu"] == [0, 0, 18, 18] and w["kv_len"] == [30, 30, 30]


def test_a_bad_free_count_moves_nothing():
    for count in (-1, 61):
        c = Cache(4, 16, 8, 60, 16)
        c.step()
        state = {k: c.d[k].clone() for k in ("kv_len", "held", "page_table")}
        c.d["free_count"].fill_(count)
        c.plan(None, [3] * 4)
        assert int(c.err.item()) == 64
        assert c.d["cu_seqlens"].tolist() == [0] * 5 and int(c.d["free_count"].item()) == count
        for k, x in state.items():
            assert torch.equal(c.d[k], x)
    # more pages going back than the list has room for (a page that two requests hold)
    c = Cache(4, 16, 8, 60, 16)
    w = c.step()
    c.d["free_count"].fill_(58)
    c.free = c.free + [0, 0]
    w = c.want(None, [0] * 4, [1] * 4)
    c.plan(None, [0] * 4, [1] * 4)
    assert int(c.err.item()) == 64 and w["err"] == 64
    assert c.d["kv_len"].tolist() == [0] * 4 and c.d["held"].tolist() == [1] * 4
    assert c.d["cu_seqlens"].tolist() == [0] * 5


@pytest.mark.parametrize("batch,max_T", [(4, 16), (40, 3000)])
def test_rows_past_the_arrays(batch, max_T):
    c = Cache(batch, 16, 200, batch * 200, max_T, max_rows=batch * max_T // 2 + 3)
    w = c.want()
    c.plan()
    c.compare(w, err=binding.GDN_DEVERR_SEQLEN)


def test_graph_replays_steps():
    c = Cache(30, 16, 20, 600, 16)
    kept = i32([0] * 30)
    p = binding.make_pages(**c.d, page_size=16, max_T=16, accepted=kept, slots=c.slots, positions=c.positions,
                           dev_err=c.err)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.gdn_plan_pages(p)
    rng = np.random.default_rng(5)
    acc = [0] * 30
    for step in range(10):
        c.slots.fill_(-3)
        c.positions.fill_(-3)
        kept.copy_(i32(acc))
        w = c.want(None, acc)
        g.replay()
        torch.cuda.synchronize()
        c.compare(w)
        c.move_on(w)
        acc = [int(rng.integers(0, 17)) for _ in range(30)]
