"""Sampled acceptance where a probability or random number is not finite: the rule of gdn.h, a draft stays if
u q(x) < p(x), taken as it stands (0 times infinity, and NaN anywhere, is no number below another)."""
import itertools

import numpy as np
import pytest
import torch

import oracle

INF, NAN = float("inf"), float("nan")
# (u, q, p, whether the draft stays)
RULE = [
    (0.5, 0.5, INF, True), (0.0, 1.0, INF, True), (0.5, 0.5, -INF, False), (0.5, 0.5, NAN, False),
    (0.5, INF, 1.0, False), (0.5, INF, INF, False), (0.0, INF, 1.0, False), (0.5, -INF, 1.0, True),
    (0.5, NAN, 1.0, False), (NAN, 0.5, INF, False), (INF, 0.5, 1.0, False), (0.5, 0.25, 0.5, True),
]
VOCAB = 5


def problem(rows):
    """A request of two rows for each (u, q, p): its draft is id 3."""
    n = len(rows)
    target = np.tile(np.float32([0.1, 0.2, 0.3, 0.25, 0.15]), (2 * n, 1))
    draft = np.tile(np.float32([0.3, 0.1, 0.1, 0.25, 0.25]), (2 * n, 1))
    u = np.zeros(2 * n, np.float32)
    for r, (x, q, p) in enumerate(rows):
        u[2 * r + 1], draft[2 * r, 3], target[2 * r, 3] = x, q, p
    return np.full(2 * n, 3, np.int32), target, draft, u, np.linspace(0, 0.999, n, dtype=np.float32), 2 * np.arange(n + 1)


def test_the_rule():
    accepted, following = oracle.accept_sample(*problem([x[:3] for x in RULE]))
    assert [a == 2 for a in accepted] == [x[3] for x in RULE]
    assert np.all((following >= 0) & (following < VOCAB))


def test_looked_up_drafts():
    ids, target, _, u, us, cu = problem([(0.5, 1.0, INF), (0.5, 1.0, NAN), (0.5, 1.0, 0.75)])
    assert list(oracle.accept_sample(ids, target, None, u, us, cu)[0]) == [2, 1, 2]


@pytest.mark.gpu
@pytest.mark.parametrize("lookup", [False, True])
def test_the_kernel_follows_it(lookup):
    from speculative_decode_gated_gb300 import binding
    values = (0.0, 0.5, 1.0, INF, -INF, NAN)
    ids, target, draft, u, us, cu = problem(list(itertools.product((0.0, 0.5, INF, NAN), values, values)))
    draft = None if lookup else draft
    want = oracle.accept_sample(ids, target, draft, u, us, cu)
    dev = [None if x is None else torch.from_numpy(x).cuda() for x in (ids, target, draft, u, us)]
    got = [torch.full((len(us),), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    binding.gdn_accept_sample(binding.make_sample(draft_ids=dev[0], target_probs=dev[1], draft_probs=dev[2], u_accept=dev[3],
                                                  u_sample=dev[4], max_T=2), *got)
    for x, y in zip(got, want):
        assert x.tolist() == y.tolist()
