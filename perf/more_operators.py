"""A speculative step beside its GDN and attention layers, as measured work: linear attention with a
decay for each head (single tokens, drafts, their commit, prompts), acceptance of sampled drafts
against the target's probabilities, and the pages, row offsets and slots of the next step.

A case is a dict of plain values; see listed().  `run` computes the operators in elementary torch
operations, or, where `own` is true, through the package's public entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
UNIT = 2.0 ** 44  # probabilities are added up in whole units of 2^-44


def _linear(name, **kw):
    c = dict(name=name, op="linear", form="step", type="bf16", batch=1, T=1, ragged=False, heads=32,
             k_heads=32, dk=128, dv=128, gates="head")
    c.update(kw)
    return c


def _sample(name, **kw):
    c = dict(name=name, op="sample", batch=1, T=5, ragged=False, vocab=32000, drafts="probs")
    c.update(kw)
    return c


def _pages(name, **kw):
    c = dict(name=name, op="pages", batch=1, T=16, ragged=False, page=16, ctx=1000, ended=0.0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token through one layer: latency
        _linear("lin_b1_t1"),
        # single tokens of 64 requests: every state read and written once
        _linear("lin_b64_t1", batch=64, gates="token"),
        # 64 requests' 16 drafts: outputs only, the states stay
        _linear("lin_verify_b64_t16", form="verify", batch=64, T=16, gates="token", k_heads=16),
        # the same requests' accepted rows into the states, uneven steps
        _linear("lin_commit_b64_t16", form="commit", batch=64, T=16, ragged=True),
        # one long prompt
        _linear("lin_prompt_b1", T=8001),
        # prompts of six requests, two value heads to a key head, a decay for each token
        _linear("lin_prompt_b6", batch=6, T=4000, ragged=True, k_heads=16, gates="token"),
        # single precision and odd sizes, as a check of a model runs it
        _linear("lin_fp32", type="fp32", batch=5, T=33, ragged=True, heads=6, k_heads=3, dk=64, dv=96,
                gates="token"),
        # one user's drafts against the target: latency
        _sample("sample_b1"),
        # 64 requests' 7 drafts
        _sample("sample_b64", batch=64, T=8, vocab=128000),
        # drafts looked up in a text (no distribution of their own), odd vocabulary, uneven steps
        _sample("sample_lookup_b200", batch=200, T=6, ragged=True, vocab=100003, drafts="lookup"),
        # the next step of 64 requests that decode with drafts
        _pages("pages_b64", batch=64, ctx=8000),
        # 1000 requests: prompt chunks of every length, some requests ended
        _pages("pages_b1000", batch=1000, T=2000, ragged=True, ctx=3000, ended=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["token", "verify", "commit", "prompt", "prompt", "fp32", "sample", "sample", "pages"])
    if kind == "sample":
        c = _sample("", batch=_log(rng, 1, 256), T=rng.randint(1, 12), ragged=rng.random() < 0.5,
                    vocab=_log(rng, 1000, 200000), drafts=rng.choice(["probs", "probs", "lookup"]))
        while c["batch"] * c["T"] * c["vocab"] > 64 * 8 * 128000:
            c["batch"] = max(1, c["batch"] * 3 // 4)
    elif kind == "pages":
        c = _pages("", batch=_log(rng, 1, 2000), T=_log(rng, 1, 2000), ragged=rng.random() < 0.5,
                   page=rng.choice([16, 32, 64, 128]), ctx=_log(rng, 1, 20000),
                   ended=rng.choice([0.0, 0.1, 0.5]))
        while c["batch"] * c["T"] > 1000 * 2000 or c["batch"] * c["ctx"] > 1000 * 3000:
            c["batch"] = max(1, c["batch"] * 3 // 4)
            c["T"] = max(1, c["T"] * 9 // 10)
    else:
        k_heads, groups = rng.choice([2, 4, 8, 16, 32]), rng.choice([1, 1, 2, 4])
        c = _linear("", batch=_log(rng, 1, 128), ragged=rng.random() < 0.5, k_heads=k_heads,
                    heads=k_heads * groups, dk=rng.choice([64, 128, 128, 128]),
                    dv=rng.choice([64, 128, 128, 128, 256]), gates=rng.choice(["head", "token"]))
        if kind == "token":
            c["ragged"] = False
        elif kind in ("verify", "commit"):
            c["form"], c["T"] = kind, rng.randint(2, 32)
        elif kind == "prompt":
            c["batch"], c["T"] = _log(rng, 1, 8), _log(rng, 50, 8000)
        else:
            c["type"], c["batch"], c["T"] = "fp32", _log(rng, 1, 8), rng.randint(1, 60)
            c["form"] = rng.choice(["step", "verify", "commit"])
            c["dk"], c["dv"] = rng.choice([32, 64, 128, 256]), rng.choice([32, 64, 96, 128, 256])
        # no drawn case costs more than the largest listed one
        while c["batch"] > 1 and (work(c)["bytes"] > 3e8 or work(c)["flops"] > 3e10):
            c["batch"] = c["batch"] * 3 // 4
        while work(c)["bytes"] > 3e8 or work(c)["flops"] > 3e10:
            c["T"] = c["T"] * 3 // 4
    del c["name"]
    return c


# ---------------------------------------------------------------- what a case's requests look like

def _parts(n, step):
    return [((r + 1) * step) % 1.0 for r in range(n)]


def _rows(case):
    """Rows of each request's step: the same whatever the seed, up to their order."""
    B, T = case["batch"], case["T"]
    if not case["ragged"]:
        return [T] * B
    new = [min(T, 1 + int(x * T)) for x in _parts(B, 0.6180339887498949)]
    new[0] = T
    return new


def _kept(case):
    """Rows of each request that its commit keeps, some of them none."""
    return [int(x * (n + 1)) for x, n in zip(_parts(case["batch"], 0.7548776662466927), _rows(case))]


def _shuffled(case, seed, *lists):
    order = list(range(case["batch"]))
    random.Random(seed).shuffle(order)
    return [[x[r] for r in order] for x in lists]


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"linear": _prepare_linear, "sample": _prepare_sample, "pages": _prepare_pages}[case["op"]](case, seed, g)
    s["case"] = case
    return s


def _offsets(new):
    return _int32([0] + [int(x) for x in np.cumsum(new)])


def _prepare_linear(case, seed, g):
    B, T, H, Hk, dk, dv = (case[k] for k in ("batch", "T", "heads", "k_heads", "dk", "dv"))
    dt = TYPES[case["type"]]
    new, kept = _shuffled(case, seed, _rows(case), _kept(case))
    n = sum(new)

    def normal(*shape):
        return torch.empty(shape, device=DEV).normal_(generator=g)

    # a projection writes queries, keys and values side by side in one row a token
    rows = normal(n, 2 * Hk * dk + H * dv)
    rows[:, Hk * dk:2 * Hk * dk] *= dk ** -0.5
    rows = rows.to(dt)
    q, k, v = rows.split((Hk * dk, Hk * dk, H * dv), 1)
    if case["gates"] == "head":  # a constant of the layer, from slow to fast over its heads
        decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, device=DEV) / H)
    else:
        decay = torch.nn.functional.logsigmoid(normal(n, H) + 3.0)
    slots = torch.randperm(B + 3, generator=g, device=DEV)[:B].to(torch.int32)
    s = dict(q=q.view(n, Hk, dk), k=k.view(n, Hk, dk), v=v.view(n, H, dv), decay=decay, slots=slots,
             pool=normal(B + 3, H, dk, dv), cu=_offsets(new), new=torch.tensor(new, device=DEV), n_tok=n,
             kept=_int32(kept), scale=1.0)
    if own:
        from speculative_decode_gated_gb300 import binding
        s["lin"] = binding.make_linear(
            q=s["q"], k=s["k"], v=s["v"], log_decay=decay, pool=s["pool"], slot_ids=slots, max_T=T,
            cu_seqlens=s["cu"] if case["ragged"] else None, scale=s["scale"])
        s["o"] = torch.empty((n, H, dv), dtype=dt, device=DEV)
    return s


def _prepare_sample(case, seed, g):
    B, V = case["batch"], case["vocab"]
    (new,) = _shuffled(case, seed, _rows(case))
    n, cu = sum(new), _offsets(new)
    logits = torch.empty((n, V), device=DEV).normal_(generator=g).mul_(3.0)
    target = torch.softmax(logits, -1)
    draft = None
    if case["drafts"] == "probs":  # a smaller model, mostly of the same mind
        draft = torch.softmax(logits.add_(torch.empty((n, V), device=DEV).normal_(generator=g), alpha=0.6), -1)
    del logits
    # the draft at row t was drawn after row t - 1; a request's first row is its last token
    ids = torch.multinomial(target if draft is None else draft, 1, generator=g).flatten().roll(1)
    s = dict(ids=ids.to(torch.int32), target=target, draft=draft, cu=cu, new=torch.tensor(new, device=DEV),
             n_tok=n, u=torch.rand(n, generator=g, device=DEV), u_next=torch.rand(B, generator=g, device=DEV))
    if own:
        from speculative_decode_gated_gb300 import binding
        s["sample"] = binding.make_sample(
            draft_ids=s["ids"], target_probs=target, draft_probs=draft, u_accept=s["u"], u_sample=s["u_next"],
            max_T=case["T"], cu_seqlens=cu if case["ragged"] else None)
        s["accepted"], s["next"] = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))
    return s


def _prepare_pages(case, seed, g):
    B, T, P, ctx = (case[k] for k in ("batch", "T", "page", "ctx"))
    old = [int((0.1 + 0.9 * x) * ctx) for x in _parts(B, 0.5698402909980532)]
    over = [x < case["ended"] for x in _parts(B, 0.4142135623730951)]
    new, kept, old, over = _shuffled(case, seed, _rows(case), _kept(case), old, over)
    held = [-(-(a + T) // P) for a in old]  # of the last step's rows too
    width = max(held) + -(-2 * T // P) + 1
    n_pages = sum(held) + sum(-(-x // P) + 1 for x in new) + 7
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    has = torch.arange(width, device=DEV)[None, :] < torch.tensor(held, device=DEV)[:, None]
    table[has] = ids[:sum(held)]
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[:n_pages - sum(held)] = ids[sum(held):]
    s = dict(table=table, free=free, count=_int32([n_pages - sum(held)]), kv_len=_int32(old), held=_int32(held),
             rows=_int32(new), kept=_int32(kept), over=_int32([int(x) for x in over]), n_pages=n_pages)
    # the lengths before and after in buffers of their own, as a step that may be tried again keeps them
    s["out"] = dict(kv_len=torch.empty_like(s["kv_len"]), held=torch.empty_like(s["held"]),
                    count=torch.empty_like(s["count"]), cu=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                    slots=torch.full((B * T,), -1, dtype=torch.int64, device=DEV),
                    positions=torch.full((B * T,), -1, dtype=torch.int32, device=DEV), table=table, free=free)
    if own:
        from speculative_decode_gated_gb300 import binding
        o = s["out"]
        s["pages"] = binding.make_pages(
            page_table=table, page_size=P, max_T=T, kv_len=s["kv_len"], held=s["held"], free_pages=free,
            free_count=s["count"], rows=s["rows"] if case["ragged"] else None, accepted=s["kept"],
            done=s["over"], kv_len_out=o["kv_len"], held_out=o["held"], free_count_out=o["count"],
            cu_seqlens=o["cu"], slots=o["slots"], positions=o["positions"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        from speculative_decode_gated_gb300 import binding
        if case["op"] == "sample":
            binding.gdn_accept_sample(s["sample"], s["accepted"], s["next"])
            return {"accepted": s["accepted"], "next": s["next"]}
        if case["op"] == "pages":
            binding.gdn_plan_pages(s["pages"])
            return s["out"]
        if case["form"] == "commit":
            binding.gdn_linear_commit(s["lin"], s["kept"])
            return {"pool": s["pool"]}
        if case["form"] == "verify":
            binding.gdn_linear_verify(s["lin"], s["o"])
            return {"o": s["o"]}
        binding.gdn_linear_step(s["lin"], s["o"])
        return {"o": s["o"], "pool": s["pool"]}
    return {"linear": _plain_linear, "sample": _plain_sample, "pages": _plain_pages}[case["op"]](s)


def _row_index(s):
    """(request, index among its rows) of each row."""
    r = torch.repeat_interleave(torch.arange(len(s["new"]), device=DEV), s["new"], output_size=s["n_tok"])
    return r, torch.arange(s["n_tok"], device=DEV) - s["cu"].long()[r]


def _plain_linear(s):
    """Blocks of up to 64 rows: within a block by products with the decays between its rows, and
    from block to block by the states before each."""
    case = s["case"]
    B, T, H, dk, dv = (case[k] for k in ("batch", "T", "heads", "dk", "dv"))
    C = min(T, 64)
    N = -(-T // C)
    r, t = _row_index(s)

    def blocks(x):  # [n_tok, heads, d] -> [B, H, N, C, d]
        y = torch.zeros((B, N * C) + x.shape[1:], dtype=x.dtype, device=DEV)
        y[r, t] = x
        return y.view(B, N, C, x.shape[1], -1).permute(0, 3, 1, 2, 4)

    decay = s["decay"].double()
    decay = decay.expand(s["n_tok"], H) if decay.dim() == 1 else decay
    keep = t < s["kept"].long()[r] if case["form"] == "commit" else torch.ones_like(t, dtype=torch.bool)
    G = blocks(torch.where(keep[:, None], decay, 0.0)[..., None])[..., 0].cumsum(-1)  # [B, H, N, C], 64 bits
    group = H // case["k_heads"]
    k = blocks(torch.where(keep[:, None, None], s["k"].float(), 0.0)).repeat_interleave(group, 1)
    v = blocks(torch.where(keep[:, None, None], s["v"].float(), 0.0))
    last = G[..., -1]
    U = torch.matmul((k * (last[..., None] - G).exp().float()[..., None]).transpose(-1, -2), v)
    # states before each block and after the last: decays between blocks times what each adds
    D = last.cumsum(-1)
    before = torch.cat((torch.zeros_like(D[..., :1]), D), -1)  # [B, H, N + 1]
    between = before[..., :, None] - D[..., None, :]
    earlier = torch.arange(N + 1, device=DEV)[:, None] > torch.arange(N, device=DEV)[None, :]
    between = between.masked_fill(~earlier, -math.inf).exp().float()
    S0 = s["pool"][s["slots"].long()]
    S = torch.matmul(between, U.reshape(B, H, N, dk * dv))
    S += before.exp().float()[..., None] * S0.view(B, H, 1, dk * dv)
    S = S.view(B, H, N + 1, dk, dv)
    out = {}
    if case["form"] != "commit":
        q = blocks(s["q"].float()).repeat_interleave(group, 1) * s["scale"]
        i = torch.arange(C, device=DEV)
        A = (G[..., :, None] - G[..., None, :]).masked_fill_(i[:, None] < i[None, :], -math.inf).exp_().float()
        A *= torch.matmul(q, k.transpose(-1, -2))
        o = torch.matmul(A, v)
        o += torch.matmul(q, S[:, :, :N]) * G.exp().float()[..., None]
        out["o"] = o.permute(0, 2, 3, 1, 4).reshape(B, N * C, H, dv)[r, t].to(s["q"].dtype)
    if case["form"] != "verify":
        s["pool"][s["slots"].long()] = S[:, :, N]
        out["pool"] = s["pool"]
    return out


def _plain_sample(s):
    case = s["case"]
    B, T, V = case["batch"], case["T"], case["vocab"]
    r, t = _row_index(s)
    ids, row = s["ids"].long(), torch.arange(s["n_tok"], device=DEV)
    before = (row - 1).clamp_(min=0)  # the row whose distributions judge a draft
    p = s["target"][before, ids].double()
    q = s["draft"][before, ids].double() if s["draft"] is not None else torch.ones_like(p)
    stay = torch.zeros((B, T), dtype=torch.int64, device=DEV)
    stay[r, t] = ((s["u"].double() * q < p) | (t == 0)).long()
    accepted = stay.cumprod(1).sum(1)
    at = s["cu"].long()[:-1] + accepted - 1  # the last row that stays
    rejected = accepted < s["new"]

    def units(x):
        return x.double().mul_(UNIT).floor_().long()

    full = units(s["target"][at])
    if s["draft"] is not None:
        less = units(s["draft"][at])
    else:
        less = torch.zeros_like(full)
        x = ids[(at + 1).clamp_(max=s["n_tok"] - 1)]
        less[torch.arange(B, device=DEV), x] = int(UNIT)
    w = torch.where(rejected[:, None], (full - less).clamp_(min=0), full)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, full)
    total = w.cumsum(1)
    W = total[:, -1]
    u = (s["u_next"].double() * 2.0 ** 31).floor().long()
    border = u * (W >> 31) + ((u * (W & 0x7FFFFFFF)) >> 31)  # u W / 2^31
    nxt = (total <= border[:, None]).sum(1)
    return {"accepted": accepted.to(torch.int32), "next": nxt.to(torch.int32)}


def _plain_pages(s):
    case, o = s["case"], s["out"]
    B, T, P = case["batch"], case["T"], case["page"]
    width, n_pages = s["table"].shape[1], s["n_pages"]
    over = s["over"] != 0
    held, count = s["held"].long(), s["count"].long()
    length = torch.where(over, 0, s["kv_len"].long() + s["kept"].long())
    rows = torch.where(over, 0, s["rows"].long())
    need = (length + rows + P - 1) // P
    back = (held - need).clamp(min=0)  # pages that go back, behind those that are free
    col = torch.arange(width, device=DEV)[None, :]
    goes = (col >= need[:, None]) & (col < held[:, None])
    place = count + back.cumsum(0)[:, None] - back[:, None] + col - need[:, None]
    free = torch.cat((s["free"], s["free"][:1]))  # and a place for what is not there
    free[torch.where(goes, place, n_pages)] = s["table"]
    available = count + back.sum()
    more = (need - held).clamp(min=0)
    until = more.cumsum(0)
    granted = until <= available
    rows = torch.where(granted, rows, 0)
    more = torch.where(granted, more, 0)
    comes = (col >= held[:, None]) & (col < (held + more)[:, None])
    taken = available - 1 - (until - (need - held).clamp(min=0))[:, None] - (col - held[:, None])
    s["table"].copy_(torch.where(comes, free[taken.clamp(0, n_pages)], s["table"]))
    s["free"].copy_(free[:n_pages])
    o["kv_len"].copy_(length)
    o["held"].copy_(torch.where(granted, need, held))
    o["count"].copy_(available - more.sum())
    ends = rows.cumsum(0)
    o["cu"][0] = 0
    o["cu"][1:] = ends
    t = torch.arange(T, device=DEV)[None, :]
    at = torch.where(t < rows[:, None], (ends - rows)[:, None] + t, B * T).flatten()
    pos = length[:, None] + t
    slot = s["table"].long().gather(1, (pos // P).clamp(max=width - 1)) * P + pos % P
    for name, x in (("slots", slot), ("positions", pos)):
        y = torch.cat((o[name], o[name][:1]))
        y[at] = x.flatten().to(y.dtype)
        o[name].copy_(y[:B * T])
    return o


# ---------------------------------------------------------------- bytes, operations, 64 bits

def work(case):
    new, B = _rows(case), case["batch"]
    n = sum(new)
    if case["op"] == "sample":
        V = case["vocab"]
        # one row of the target's probabilities a request, and of the draft's where a draft falls
        # (about four in five of them stay)
        rows = sum(2.0 - 0.8 ** (x - 1) for x in new) if case["drafts"] == "probs" else B
        return {"bytes": 4 * V * rows + 20 * n + 12 * B, "flops": 3 * V * rows}
    if case["op"] == "pages":
        pages = sum(-(-x // case["page"]) for x in new)
        return {"bytes": 12 * n + 8 * pages + 32 * B, "flops": 4 * n}
    H, Hk, dk, dv = (case[k] for k in ("heads", "k_heads", "dk", "dv"))
    size = 2 if case["type"] == "bf16" else 4
    if case["form"] == "commit":
        kept = _kept(case)
        n, states = sum(kept), 2 * sum(x > 0 for x in kept)
        per_row = (Hk * dk + H * dv) * size
    else:
        states = B * (2 if case["form"] == "step" else 1)
        per_row = 2 * (Hk * dk + H * dv) * size
    per_row += 4 * H if case["gates"] == "token" else 0
    return {"bytes": n * per_row + 4 * states * H * dk * dv, "flops": 4 * n * H * dk * dv}


def exact(case, seed):
    if case["op"] != "linear":
        return None  # whole numbers
    s = prepare(case, seed)
    B, H, dk, dv = (case[k] for k in ("batch", "heads", "dk", "dv"))
    new, cu, kept = s["new"].tolist(), s["cu"].tolist(), s["kept"].tolist()
    if case["form"] == "commit":
        new = kept
    head = torch.arange(H, device=DEV) // (H // case["k_heads"])
    state = s["pool"][s["slots"].long()].double()
    o = torch.zeros((s["n_tok"], H, dv), dtype=torch.float64, device=DEV)
    decay = s["decay"].double()
    order = sorted(range(B), key=lambda r: -new[r])  # longest first: a step takes the first few
    state = state[order]
    for t in range(max(new)):
        live = sum(1 for x in new if x > t)
        rows = torch.tensor([cu[r] + t for r in order[:live]], device=DEV) if B > 1 else slice(t, t + 1)
        lam = decay.exp()[None] if decay.dim() == 1 else decay[rows].exp()
        k, v = s["k"][rows][:, head].double(), s["v"][rows].double()
        S = state[:live] * lam[:, :, None, None] + k[..., :, None] * v[..., None, :]
        state[:live] = S
        if case["form"] != "commit":
            o[rows] = (s["q"][rows][:, head].double()[..., None, :] @ S)[..., 0, :] * s["scale"]
    pool = s["pool"].double()
    pool[s["slots"].long()[order]] = state
    return {"step": {"o": o, "pool": pool}, "verify": {"o": o}, "commit": {"pool": pool}}[case["form"]]
