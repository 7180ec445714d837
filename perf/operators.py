"""The attention layers of a hybrid verification step, as measured work: rotary positions with the
append to a paged cache, and attention of a chunk of new tokens over that cache (all of it, or a
sliding window with a few first tokens that stay visible).

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


def _rope(name, **kw):
    c = dict(name=name, op="rope", type="bf16", batch=1, T=1, ragged=False, q_heads=32, kv_heads=8,
             hd=128, page=16, ctx=1000, spread=True, rot=128, interleaved=False, base=10000.0,
             scaling="none", factor=1.0)
    c.update(kw)
    return c


def _attn(name, **kw):
    c = dict(name=name, op="attn", type="bf16", batch=1, T=1, ragged=False, q_heads=32, kv_heads=8,
             hd=128, page=16, ctx=1000, spread=True, window=0, sinks=0, lse=False)
    c.update(kw)
    return c


def listed():
    return [
        # one user's next token: nothing but latency
        _rope("rope_b1_t1", ctx=1000),
        # a verification step of 64 requests with 16 drafts each, positions scaled to long contexts
        _rope("rope_b64_t16_yarn", batch=64, T=16, ctx=100000, scaling="yarn", factor=32.0),
        # a prompt chunk of four requests; pairs side by side, a quarter of a wide head rotated
        _rope("rope_prompt_part", batch=4, T=2000, ragged=True, q_heads=16, kv_heads=4, hd=256,
              page=64, ctx=5000, rot=64, interleaved=True),
        # single precision, as a check of a model runs it
        _rope("rope_fp32", type="fp32", batch=8, T=33, ragged=True, q_heads=16, kv_heads=16, hd=64,
              page=32, ctx=30000, rot=64, scaling="linear", factor=4.0),
        # one user's next token over a short context: latency
        _attn("attn_b1_t1", ctx=1000),
        # single tokens of 64 requests, contexts of every length up to 8 thousand
        _attn("attn_b64_t1", batch=64, ctx=8191),
        # the same requests verifying 16 drafts
        _attn("attn_b64_t16", batch=64, T=16, ctx=4000, lse=True),
        # one request's 16 drafts over a long document, heads of 64
        _attn("attn_b1_t16_long", T=16, hd=64, q_heads=64, page=64, ctx=130001),
        # a prompt chunk of two requests over what they already hold
        _attn("attn_prompt", batch=2, T=4001, ctx=6007, spread=False, page=64),
        # ragged drafts of 128 requests in a window with sinks
        _attn("win_b128_ragged", batch=128, T=16, ragged=True, q_heads=32, kv_heads=4, ctx=20000,
              window=1024, sinks=4, page=32),
        # a prompt chunk through a windowed layer
        _attn("win_prompt", T=8000, q_heads=64, hd=64, ctx=900, spread=False, window=512, sinks=4,
              lse=True),
        # single precision, an odd number of heads to a key head, empty pages at the ends
        _attn("attn_fp32", type="fp32", batch=5, T=7, ragged=True, q_heads=15, kv_heads=3, hd=64,
              ctx=777, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "decode", "drafts", "drafts", "prompt", "window", "fp32"])
    groups = rng.choice([1, 2, 4, 5, 8, 16])
    hd = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8]) if groups > 4 else rng.choice([2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    heads = dict(q_heads=groups * kv_heads, kv_heads=kv_heads, hd=hd, page=page)
    if kind == "rope":
        batch = _log(rng, 1, 128)
        c = _rope("", batch=batch, T=min(_log(rng, 1, 4000), max(1, 8000 // batch)),
                  ragged=rng.random() < 0.5, ctx=_log(rng, 1, 120000),
                  rot=rng.choice([hd, hd, hd // 2, hd // 4]), interleaved=rng.random() < 0.5,
                  base=rng.choice([10000.0, 500000.0]),
                  scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                  factor=rng.choice([2.0, 8.0, 32.0]), type=rng.choice(["bf16", "bf16", "fp32"]),
                  **heads)
    else:
        c = _attn("", batch=_log(rng, 1, 128), ctx=_log(rng, 1, 40000),
                  ragged=rng.random() < 0.5, spread=rng.random() < 0.7, lse=rng.random() < 0.3,
                  **heads)
        if kind == "decode":
            c["T"], c["ragged"] = 1, False
        elif kind == "drafts":
            c["T"] = rng.randint(2, 32)
        elif kind == "prompt":
            c["T"], c["batch"], c["hd"] = _log(rng, 100, 8000), _log(rng, 1, 8), min(hd, 128)
        elif kind == "window":
            c["T"], c["window"], c["sinks"] = _log(rng, 1, 2000), _log(rng, 32, 8000), rng.choice([0, 4, 20])
            c["hd"] = min(hd, 128)
        else:
            c["type"], c["T"], c["batch"] = "fp32", rng.randint(1, 48), _log(rng, 1, 8)
            c["ctx"] = min(c["ctx"], 4000)
    del c["name"]  # no drawn case costs more than the largest listed one
    while c["op"] == "rope" and work(c)["bytes"] > 5e8:
        c["T"], c["batch"] = max(1, c["T"] // 2), max(1, c["batch"] * 3 // 4)
    if c["op"] == "attn":
        scores, cache = (2e9, 3e8) if c["type"] == "bf16" else (2e7, 2e7)

        def over():
            n = c["ctx"] + c["T"]
            return (c["batch"] * c["q_heads"] * c["T"] * n > scores
                    or c["batch"] * c["kv_heads"] * c["hd"] * n > cache)

        while over() and c["batch"] > 1:
            c["batch"] = c["batch"] * 3 // 4
        while over():
            c["T"], c["ctx"] = max(1, c["T"] * 4 // 5), max(1, c["ctx"] * 4 // 5)
    return c


# ---------------------------------------------------------------- what a case's requests look like

def _lengths(case):
    """(new tokens, tokens before) of each request: the same whatever the seed, up to their order."""
    B, T, ctx = case["batch"], case["T"], case["ctx"]
    part = [((r + 1) * 0.6180339887498949) % 1.0 for r in range(B)]
    new = [1 + int(part[r] * T) if case["ragged"] else T for r in range(B)]
    if case["ragged"]:
        new = [min(T, n) for n in new]
        new[0] = T
    part = [((r + 1) * 0.7548776662466927) % 1.0 for r in range(B)]
    old = [int((0.25 + 0.75 * part[r]) * ctx) if case["spread"] else ctx for r in range(B)]
    old[B // 2] = ctx
    return new, old


def _frequencies(case):
    """The angle a position adds to each pair, and the factor on cosine and sine (YaRN's)."""
    rot, base, s = case["rot"], case["base"], case["factor"]
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / s, 1.0
    if case["scaling"] == "ntk":
        return (base * s ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if case["scaling"] == "yarn":
        turns = 4096 * f / (2 * math.pi)  # of a pair over the length the model was trained on
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / s * (1 - keep), 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, old = _lengths(case)
    order = list(range(case["batch"]))
    random.Random(seed).shuffle(order)
    new, old = [new[r] for r in order], [old[r] for r in order]
    B, Hq, Hkv, hd, P = (case[k] for k in ("batch", "q_heads", "kv_heads", "hd", "page"))
    dt = TYPES[case["type"]]
    n_tok, rope = sum(new), case["op"] == "rope"
    width = -(-max(a + b for a, b in zip(new, old)) // P)
    # pages: those the new tokens touch (rope), or all that the request holds
    first = [(b // P if rope else 0) for b in old]
    last = [(a + b - 1) // P for a, b in zip(new, old)]
    n_pages = sum(z - y + 1 for y, z in zip(first, last)) + 3
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.zeros((B, width), dtype=torch.int32), 0
    for r in range(B):
        k = last[r] - first[r] + 1
        table[r, first[r]:last[r] + 1] = ids[at:at + k]
        at += k
    kp = torch.empty((n_pages, Hkv, P, hd), dtype=dt, device=DEV).normal_(generator=g)
    vp = torch.empty((n_pages, Hkv, P, hd), dtype=dt, device=DEV).normal_(generator=g)
    cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV)
    s = dict(case=case, n_tok=n_tok, k_pages=kp, v_pages=vp, table=table.to(DEV), cu=cu,
             kv_len=torch.tensor(old, dtype=torch.int32, device=DEV),
             new=torch.tensor(new, device=DEV), width=width)
    if rope:
        # a projection writes queries, keys and values side by side in one row a token
        rows = torch.empty((n_tok, Hq + 2 * Hkv, hd), dtype=dt, device=DEV).normal_(generator=g)
        s["q"], s["k"], s["v"] = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        f, s["mscale"] = _frequencies(case)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float32, device=DEV)
    else:
        # scores spread over a few units, as a trained layer's do
        s["q"] = (torch.empty((n_tok, Hq, hd), device=DEV).normal_(generator=g) * 2.0).to(dt)
        s["scale"] = 1.0 / math.sqrt(hd)
    if own:
        from speculative_decode_gated_gb300 import binding
        s["attn"] = binding.make_attn(
            q_heads=Hq, k_pages=kp, v_pages=vp, page_table=s["table"], kv_len=s["kv_len"],
            max_T=case["T"], cu_seqlens=cu if case["ragged"] else None, n_tok=n_tok,
            window=case.get("window", 0), sinks=case.get("sinks", 0), scale=s.get("scale"))
        s["out"] = torch.empty((n_tok, Hq, hd), dtype=dt, device=DEV)
        if rope:
            s["rope"] = binding.make_rope(inv_freq=s["inv_freq"], interleaved=case["interleaved"],
                                          mscale=s["mscale"])
        else:
            s["lse"] = torch.empty((n_tok, Hq), device=DEV) if case["lse"] else None
            s["workspace"] = binding.paged_attn_workspace(s["attn"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if s["case"]["op"] == "rope":
        if own:
            from speculative_decode_gated_gb300 import binding
            binding.gdn_rope_append(s["attn"], s["rope"], s["q"], s["k"], s["v"], s["out"])
            return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        return _plain_rope(s)
    if own:
        from speculative_decode_gated_gb300 import binding
        binding.gdn_paged_attn(s["attn"], s["q"], s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"o": s["out"], "lse": s["lse"]} if s["case"]["lse"] else {"o": s["out"]}
    return _plain_attn(s)


def _rows(s):
    """(request, index among its new tokens) of each row."""
    r = torch.repeat_interleave(torch.arange(len(s["new"]), device=DEV), s["new"],
                                output_size=s["n_tok"])
    return r, torch.arange(s["n_tok"], device=DEV) - s["cu"].long()[r]


def _plain_rope(s):
    case, (r, t) = s["case"], _rows(s)
    rot, P = case["rot"], case["page"]
    pos = s["kv_len"].long()[r] + t
    # 32 bits cannot hold a long context's angle: it is reduced to one turn first
    angle = torch.remainder(pos.double()[:, None] * s["inv_freq"].double(), 2 * math.pi).float()
    cos = (angle.cos() * s["mscale"])[:, None, :]
    sin = (angle.sin() * s["mscale"])[:, None, :]

    def turned(x):
        y = x.float()
        a, b = ((y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"]
                else (y[..., :rot // 2], y[..., rot // 2:rot]))
        a, b = a * cos - b * sin, a * sin + b * cos
        z = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((z, y[..., rot:]), -1).to(x.dtype)

    page, row = s["table"].long()[r, pos // P], pos % P
    s["k_pages"][page, :, row] = turned(s["k"])
    s["v_pages"][page, :, row] = s["v"]
    return {"q": turned(s["q"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attn(s):
    case, (r, t) = s["case"], _rows(s)
    B, T, Hq, Hkv, hd = (case[k] for k in ("batch", "T", "q_heads", "kv_heads", "hd"))
    G, L = Hq // Hkv, s["width"] * case["page"]
    q = torch.zeros((B, T, Hq, hd), device=DEV)
    q[r, t] = s["q"].float()
    q = q.view(B, T, Hkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, hd)

    def gathered(pages):
        return pages[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, Hkv, L, hd).float()

    x = torch.matmul(q, gathered(s["k_pages"]).transpose(-1, -2)).mul_(s["scale"])
    p = (s["kv_len"].long()[:, None] + torch.arange(T, device=DEV))[:, :, None]
    j = torch.arange(L, device=DEV)
    seen = j <= p
    if case["window"]:
        seen &= (j > p - case["window"]) | (j < case["sinks"])
    x.view(B, Hkv, T, G, L).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, gathered(s["v_pages"])).div_(total)
    o = o.view(B, Hkv, T, G, hd).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, hd)[r, t]
    out = {"o": o.to(s["q"].dtype)}
    if case["lse"]:
        lse = (m + total.log()).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
        out["lse"] = lse[r, t]
    return out


# ---------------------------------------------------------------- bytes, operations, 64 bits

def work(case):
    new, old = _lengths(case)
    size = 2 if case["type"] == "bf16" else 4
    Hq, Hkv, hd, n = case["q_heads"], case["kv_heads"], case["hd"], sum(new)
    if case["op"] == "rope":
        return {"bytes": 2 * n * (Hq + 2 * Hkv) * hd * size, "flops": 3 * n * (Hq + Hkv) * case["rot"]}
    W, sinks, keys, pairs = case["window"], case["sinks"], 0, 0
    for a, b in zip(new, old):
        if not W:
            keys += a + b
            pairs += a * b + a * (a + 1) // 2
            continue
        start = max(0, b - W + 1)  # the first position that the first row's window holds
        keys += a + b - start + min(sinks, start)
        p = np.arange(b, a + b, dtype=np.int64)
        low = np.maximum(0, p - W + 1)
        pairs += int((p + 1 - low + np.minimum(sinks, low)).sum())
    return {"bytes": 2 * n * Hq * hd * size + 2 * keys * Hkv * hd * size + (4 * n * Hq if case["lse"] else 0),
            "flops": 4 * hd * Hq * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    new, old = _lengths(case)
    cu, kv_len = s["cu"].tolist(), s["kv_len"].tolist()
    B, Hq, Hkv, hd, P = (case[k] for k in ("batch", "q_heads", "kv_heads", "hd", "page"))
    if case["op"] == "rope":
        half = case["rot"] // 2
        q, kp, vp = s["q"].double(), s["k_pages"].double(), s["v_pages"].double()
        k = s["k"].double()
        pos = torch.cat([torch.arange(kv_len[r], kv_len[r] + cu[r + 1] - cu[r]) for r in range(B)]).to(DEV)
        turn = torch.polar(torch.full((s["n_tok"], half), float(s["mscale"]), dtype=torch.float64, device=DEV),
                           pos.double()[:, None] * s["inv_freq"].double()[None, :])
        for x in (q, k):
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
                z = torch.complex(x[:, :, a], x[:, :, b]) * turn[:, i:i + 1]
                x[:, :, a], x[:, :, b] = z.real.clone(), z.imag.clone()
        for r in range(B):
            p = pos[cu[r]:cu[r + 1]]
            for c in torch.unique(p // P).tolist():
                rows = torch.nonzero(p // P == c).flatten()
                at = int(s["table"][r, c])
                kp[at, :, p[rows] % P] = k[cu[r] + rows].transpose(0, 1)
                vp[at, :, p[rows] % P] = s["v"][cu[r] + rows].double().transpose(0, 1)
        return {"q": q, "k_pages": kp, "v_pages": vp}
    G, W = Hq // Hkv, case["window"]
    o = torch.zeros((s["n_tok"], Hq, hd), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["n_tok"], Hq), dtype=torch.float64, device=DEV)
    for r in range(B):
        T, end = cu[r + 1] - cu[r], kv_len[r] + cu[r + 1] - cu[r]
        pages = s["table"][r, :-(-end // P)].long()
        j = torch.arange(end, device=DEV)[None, :]
        p = torch.arange(kv_len[r], end, device=DEV)[:, None]
        hidden = j > p
        if W:
            hidden |= (p - j >= W) & (j >= case["sinks"])
        for h in range(Hkv):
            k = s["k_pages"][pages, h].reshape(-1, hd)[:end].double()
            v = s["v_pages"][pages, h].reshape(-1, hd)[:end].double()
            for g in range(h * G, (h + 1) * G):
                x = s["q"][cu[r]:cu[r + 1], g].double() @ k.T * s["scale"]
                x[hidden] = -math.inf
                top = torch.logsumexp(x, -1)
                lse[cu[r]:cu[r + 1], g] = top
                o[cu[r]:cu[r + 1], g] = torch.exp(x - top[:, None]) @ v
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
