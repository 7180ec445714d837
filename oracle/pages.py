"""The pages of a paged cache's next step (CPU oracle), request by request with Python lists.

TEST INFRASTRUCTURE, like the rest of this package: only `tests/` and
`__graft_entry__.smoke()` use it.

Parity unpinned: none.  Pinned by `tests/test_step_oracles.py`.
"""
from __future__ import annotations

SEQLEN, ACCEPTED, KV_LEN, PAGE, NO_PAGES = 4, 2, 32, 64, 256


def plan_pages(kv_len, held, free, table, page, max_T, n_pages=None, rows=None, accepted=None, done=None):
    """free: the free list; table: a list of page ids per request, max_pages long.

    Returns a dict: kv_len, held, free (the list), table, cu, slots, positions, err."""
    B, width = len(kv_len), len(table[0]) if table else 0
    table = [list(t) for t in table]
    stack, err = list(free), 0
    lengths, want, need, stays = [], [], [], []
    for r in range(B):
        over = bool(done[r]) if done is not None else False
        a = int(accepted[r]) if accepted is not None else 0
        T = int(rows[r]) if rows is not None else max_T
        bad = 0
        if not 0 <= held[r] <= width or (not over and kv_len[r] < 0):
            bad |= KV_LEN
        if not over and not bad and (a < 0 or kv_len[r] + a > held[r] * page):
            bad |= ACCEPTED
        if not over and not 0 <= T <= max_T:
            bad |= SEQLEN
        err |= bad
        if bad:
            lengths.append(kv_len[r])
            want.append(0)
            need.append(held[r])
            continue
        length, T = (0, 0) if over else (kv_len[r] + a, T)
        if length + T > width * page:
            err |= KV_LEN
            T = 0
        lengths.append(length)
        want.append(T)
        need.append(-(-(length + T) // page))
    going = [table[r][c] for r in range(B) for c in range(need[r], held[r])]
    if n_pages is not None and len(stack) + len(going) > n_pages:
        return dict(kv_len=list(kv_len), held=list(held), free=stack, table=table, cu=[0] * (B + 1),
                    slots=[], positions=[], err=err | PAGE)
    stack += going
    available, asked = len(stack), 0
    out_held, cu, slots, positions = [], [0], [], []
    for r in range(B):
        more = max(need[r] - held[r], 0)
        asked += more
        T = want[r]
        if more and asked > available:
            err |= NO_PAGES
            out_held.append(held[r])
            T = 0
        else:
            for c in range(held[r], held[r] + more):
                table[r][c] = stack.pop()
            out_held.append(need[r])
        cu.append(cu[-1] + T)
        for p in range(lengths[r], lengths[r] + T):
            slots.append(table[r][p // page] * page + p % page)
            positions.append(p)
    return dict(kv_len=lengths, held=out_held, free=stack, table=table, cu=cu, slots=slots,
                positions=positions, err=err)
