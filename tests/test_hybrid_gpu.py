"""A hybrid model's verification steps end to end (examples/hybrid_step.py): GDN layers and
attention layers over one set of requests, drafts accepted on the device, states committed and
cache lengths moved.  Decoding with drafts must give the tokens of decoding one by one: in
float32 the two runs' logits differ by rounding only, far less than the gap between the
first and the second choice of a random model."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "hybrid_step.py")


def example():
    spec = importlib.util.spec_from_file_location("hybrid_step", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("window,sinks", [(0, 0), (12, 2)])
def test_drafts_do_not_change_the_tokens(window, sinks):
    m = example()
    model = m.HybridModel(dtype=torch.float32, window=window, sinks=sinks)
    first = torch.arange(3, dtype=torch.int32, device="cuda") + 1
    plain, steps, kept = m.decode(model, 3, first, 40)
    assert steps == 40 and kept == 1.0
    g = torch.Generator(device="cuda").manual_seed(1)
    wrong = torch.rand(plain.shape, generator=g, device="cuda") < 0.25
    drafts = torch.where(wrong, (plain + 1) % 512, plain)
    for rows in (2, 5, 17):
        spec, steps, kept = m.decode(model, 3, first, 40, rows, drafts)
        assert torch.equal(spec, plain)
        assert steps < 40 and kept > 1.0


def test_bf16_rows_at_once_and_one_by_one():
    # Single rows and nine at once go through different kernels.  Each of the five layers rounds
    # its output to bfloat16 (2^-9 of it, twice in its products), so logits of unit variance
    # differ by some 5^(1/2) 2^-7 in the mean and, over 2^14 of them, by some five times that.
    m = example()
    model = m.HybridModel()
    tokens = torch.randint(0, 512, (4, 9), dtype=torch.int32, device="cuda",
                           generator=torch.Generator(device="cuda").manual_seed(3))
    at_once = m.Session(model, 4, 9, 32).logits(tokens)
    s, rows = m.Session(model, 4, 1, 32), []
    for t in range(9):
        rows.append(s.logits(tokens[:, t:t + 1].contiguous()))
        s.accepted.fill_(1)
        for p in s.problems.values():
            m.binding.gdn_commit(p, s.accepted)
        s.kv_len += 1
    diff = (at_once - torch.cat(rows, 1)).abs()
    assert float(diff.square().mean().sqrt()) <= 0.02 * 2.5
    assert float(diff.max()) <= 0.02 * 2.5 * 6
