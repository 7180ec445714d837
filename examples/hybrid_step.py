"""Greedy speculative decoding of a small hybrid model: Gated DeltaNet layers and attention layers.

A model with random weights (no checkpoint is needed) whose layers alternate: GDN layers keep a
recurrent state per request and head in a pool, attention layers keep keys and values in pages.
One step of all requests:

  1. every layer runs the step's rows (the last accepted token and the drafts after it):
     gdn_verify, which leaves the state as it is, or gdn_rope_append and gdn_paged_attn;
  2. gdn_accept_prefix compares the drafts with the model's own choices, on the device;
  3. gdn_commit replays the accepted rows into the states, and kv_len moves past the accepted
     places: the next step overwrites the rejected ones.

    python examples/hybrid_step.py [--tokens 64] [--drafts 8] [--bf16]

Drafts come from a run that decodes one token a step, with some of them replaced, so the
accepted lengths vary; at the end the two runs' tokens are compared.  They agree in float32;
in bfloat16 a random model's close calls fall either way, and the drafts fit no longer from
the first one on.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from speculative_decode_gated_gb300 import binding, staging  # noqa: E402


class HybridModel:
    """Weights of `layers` ("gdn" or "attn"), each a normalised input, a projection to the
    layer's rows, the layer, and a projection back that is added to the residual."""

    def __init__(self, layers=("gdn", "gdn", "attn", "gdn", "attn"), width=256, heads=2, dim=128,
                 q_heads=4, kv_heads=1, vocab=512, window=0, sinks=0, dtype=torch.bfloat16, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            w = torch.empty((rows, cols), device=device).normal_(generator=g) * rows ** -0.5
            return w.to(dtype)

        self.layers, self.dtype, self.device = layers, dtype, torch.device(device)
        self.heads, self.dim, self.q_heads, self.kv_heads = heads, dim, q_heads, kv_heads
        self.window, self.sinks = window, sinks
        self.embed = torch.empty((vocab, width), device=device).normal_(generator=g).to(dtype)
        self.head = weight(width, vocab)
        self.w_in, self.w_out = [], []
        for kind in layers:
            cols = heads * (3 * dim + 2) if kind == "gdn" else (q_heads + 2 * kv_heads) * dim
            self.w_in.append(weight(width, cols))
            self.w_out.append(weight((heads if kind == "gdn" else q_heads) * dim, width))
        inv_freq, mscale = staging.rope_frequencies(dim, scaling="yarn", factor=4.0, device=device)
        self.rope = binding.make_rope(inv_freq=inv_freq, mscale=mscale)


def norm(x, n=None):
    y = x.float()
    return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) if n is None else \
        y / (y.norm(dim=-1, keepdim=True) + 1e-6)


class Session:
    """The states and caches of `batch` requests, and steps of `rows` rows each."""

    def __init__(self, model: HybridModel, batch: int, rows: int, max_tokens: int, page: int = 16):
        self.m, self.batch, self.rows = model, batch, rows
        dev, dt = model.device, model.dtype
        width = -(-(max_tokens + rows) // page)
        self.slot_ids = torch.arange(batch, dtype=torch.int32, device=dev)
        self.accepted = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.kv_len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.dev_err = torch.zeros(1, dtype=torch.int32, device=dev)
        # request r's page i is page i * batch + r: any table will do
        self.table = (torch.arange(width, dtype=torch.int32, device=dev)[None, :] * batch
                      + self.slot_ids[:, None]).contiguous()
        self.pools, self.attns, self.workspaces, self.problems = {}, {}, {}, {}
        for i, kind in enumerate(model.layers):
            if kind == "gdn":
                self.pools[i] = staging.new_pool(batch, model.heads, model.dim, model.dim, dev, "zero")
                continue
            pages = [torch.empty((width * batch, model.kv_heads, page, model.dim), dtype=dt, device=dev)
                     for _ in range(2)]
            self.attns[i] = binding.make_attn(
                q_heads=model.q_heads, k_pages=pages[0], v_pages=pages[1], page_table=self.table,
                kv_len=self.kv_len, max_T=rows, window=model.window, sinks=model.sinks,
                dev_err=self.dev_err)
            self.workspaces[i] = binding.paged_attn_workspace(self.attns[i])

    def _gdn(self, i, x):
        m, n = self.m, x.shape[0]
        y = (x @ m.w_in[i]).float().view(n, m.heads, 3 * m.dim + 2)
        q, k, v, gate = y.split((m.dim, m.dim, m.dim, 2), -1)
        q, k, v = (t.to(m.dtype).contiguous() for t in (norm(q, 1) * m.dim ** -0.5, norm(k, 1), v))
        alpha, beta = torch.sigmoid(gate[..., 0] + 3.0), torch.sigmoid(gate[..., 1])
        o = torch.empty((n, m.heads, m.dim), device=x.device)
        self.problems[i] = binding.make_problem(
            q=q, k=k, v=v, alpha=alpha.contiguous(), beta=beta.contiguous(), pool=self.pools[i],
            slot_ids=self.slot_ids, max_T=self.rows, dev_err=self.dev_err)
        binding.gdn_verify(self.problems[i], o)
        return norm(o).to(m.dtype).view(n, -1)

    def _attention(self, i, x):
        m, n = self.m, x.shape[0]
        y = (x @ m.w_in[i]).view(n, m.q_heads + 2 * m.kv_heads, m.dim)
        q, k, v = y.split((m.q_heads, m.kv_heads, m.kv_heads), 1)  # slices of one projection
        turned, o = (torch.empty((n, m.q_heads, m.dim), dtype=m.dtype, device=x.device)
                     for _ in range(2))
        binding.gdn_rope_append(self.attns[i], m.rope, q, k, v, turned)
        binding.gdn_paged_attn(self.attns[i], turned, o, workspace=self.workspaces[i])
        return o.view(n, -1)

    def logits(self, tokens):
        """tokens: [batch, rows] ids to feed; [batch, rows, vocab] float32."""
        m = self.m
        x = m.embed[tokens.reshape(-1).long()].float()
        for i, kind in enumerate(m.layers):
            y = norm(x).to(m.dtype)
            x = x + ((self._gdn if kind == "gdn" else self._attention)(i, y) @ m.w_out[i]).float()
        return (norm(x).to(m.dtype) @ m.head).float().view(self.batch, self.rows, -1)

    def step(self, tokens, active):
        """Feeds tokens [batch, rows] (the last accepted one, then drafts), keeps the rows that the
        model agrees with, none of a request that is not active (int32 [batch], 1 or 0);
        (accepted [batch], the model's choice after each row)."""
        choice = self.logits(tokens).argmax(-1).to(torch.int32)
        # row t's own target is the choice after row t - 1; the first row is always kept
        target = torch.cat((tokens[:, :1], choice[:, :-1]), 1).contiguous()
        binding.gdn_accept_prefix(tokens.contiguous().view(-1), target.view(-1), self.accepted,
                                  self.rows, dev_err=self.dev_err)
        self.accepted *= active
        for p in self.problems.values():
            binding.gdn_commit(p, self.accepted)
        self.kv_len += self.accepted
        return self.accepted, choice


def decode(model, batch, first, tokens, rows=1, drafts=None):
    """Greedy ids [batch, tokens] after `first` [batch]; drafts [batch, tokens]: what to propose.
    Returns (ids, steps, mean accepted rows)."""
    s = Session(model, batch, rows, tokens + rows)
    out = torch.zeros((batch, tokens + rows), dtype=torch.int32, device=model.device)
    done = torch.zeros(batch, dtype=torch.long, device=model.device)  # ids known
    last, steps, kept = first.clone(), 0, 0
    lanes = torch.arange(rows, device=model.device)
    padded = None if drafts is None else torch.nn.functional.pad(drafts, (0, 2 * rows))
    while int(done.min()) < tokens:
        feed = last[:, None].repeat(1, rows)
        if rows > 1:
            feed[:, 1:] = torch.gather(padded, 1, done[:, None] + lanes[None, :-1])
        accepted, choice = s.step(feed, (done < tokens).to(torch.int32))
        a = accepted.long()
        steps, kept = steps + 1, kept + float(a.float().mean())
        r, t = torch.nonzero(lanes[None, :] < a[:, None], as_tuple=True)
        out[r, done[r] + t] = choice[r, t]  # the choices after the accepted rows are the next ids
        newest = torch.gather(choice, 1, (a - 1).clamp(min=0)[:, None]).flatten()
        last = torch.where(a > 0, newest, last)
        done = done + a
    if int(s.dev_err.item()):
        raise RuntimeError(f"device error word {int(s.dev_err.item())}")
    return out[:, :tokens], steps, kept / steps


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--drafts", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--bf16", action="store_true")
    a = ap.parse_args()
    model = HybridModel(dtype=torch.bfloat16 if a.bf16 else torch.float32)
    first = torch.arange(a.batch, dtype=torch.int32, device="cuda") + 1
    plain, steps, _ = decode(model, a.batch, first, a.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    wrong = torch.rand(plain.shape, generator=g, device="cuda") < 0.2
    drafts = torch.where(wrong, (plain + 1) % 512, plain)
    spec, spec_steps, kept = decode(model, a.batch, first, a.tokens, 1 + a.drafts, drafts)
    same = float((spec == plain).float().mean())
    print(f"one by one: {steps} steps; with {a.drafts} drafts: {spec_steps} steps, "
          f"{kept:.2f} rows kept a step; {100 * same:.1f}% of the ids agree")


if __name__ == "__main__":
    main()
