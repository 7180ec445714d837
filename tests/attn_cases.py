"""Inputs of the attention tests: a paged cache whose unused places hold NaN, and the
calls of the binding beside the float64 oracle, with tolerances derived from the
number formats.

Tolerance of one output o = sum_j w_j v_j.  bf16: the result is rounded once,
at most 2^-8 |o| (half a unit in the last place of an 8-bit significand), and the weights
are rounded to bf16 before their product, at most 2^-8 sum_j w_j |v_j|; a float32
score of head_dim products of a few units is off by less than 2^-12, so the
weights by less than 2^-11 of themselves each way.  float32: the score's
error, below head_dim 2^-24 sum |q k| scale < 2^-14 for these inputs, twice
(numerator and denominator)."""
import numpy as np
import torch

import oracle
from speculative_decode_gated_gb300 import binding
from speculative_decode_gated_gb300.inputs import bf16_bits

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def rounded(x, dtype):
    """float32 values that dtype holds exactly."""
    x = np.ascontiguousarray(x, np.float32)
    if dtype == "bf16":
        return torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    return x


def to_dev(x, dtype, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(TYPES[dtype]).to(device)


class Case:
    """One step of some requests over a paged cache.

    new, old: tokens of the step and cached before it, per request.  The cache already holds
    the step's own keys and values.  Pages are dealt in random order; every place that
    no row of its request sees, and every page that no request has, holds NaN (or
    the value `fill`)."""

    def __init__(self, *, new, old, q_heads, kv_heads, hd, page=16, dtype="bf16", window=0,
                 sinks=0, seed=0, scale=None, fill=np.nan, qscale=2.0):
        rng = np.random.default_rng(seed)
        self.new, self.old, self.dtype = list(new), list(old), dtype
        self.q_heads, self.kv_heads, self.hd, self.page = q_heads, kv_heads, hd, page
        self.window, self.sinks = window, sinks
        self.scale = hd ** -0.5 if scale is None else scale
        self.B = len(new)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_tok = int(self.cu[-1])
        need = [-(-(a + b) // page) for a, b in zip(new, old)]
        self.width = max(need + [1]) + 1
        n_pages = sum(need) + 3
        ids = rng.permutation(n_pages)
        self.table = np.full((self.B, self.width), -5, np.int32)  # unused entries: never read
        shape = (n_pages, kv_heads, page, hd)
        self.k = np.full(shape, fill, np.float32)
        self.v = np.full(shape, fill, np.float32)
        at = 0
        for r in range(self.B):
            self.table[r, :need[r]] = ids[at:at + need[r]]
            at += need[r]
            n = self.old[r] + self.new[r]
            kr = rounded(rng.standard_normal((n, kv_heads, hd)), dtype)
            vr = rounded(rng.standard_normal((n, kv_heads, hd)), dtype)
            if window and self.new[r]:  # a windowed cache may have lost what no row sees
                c = np.arange(n)
                seen = (c > self.old[r] - window) | (c < sinks)
                kr[~seen] = fill
                vr[~seen] = fill
                gone = [i for i in range(need[r]) if not seen[i * page:(i + 1) * page].any()]
                self.table[r, gone] = -7
            for c in range(n):
                p = self.table[r, c // page]
                if p >= 0:
                    self.k[p, :, c % page] = kr[c]
                    self.v[p, :, c % page] = vr[c]
        self.q = rounded(qscale * rng.standard_normal((self.n_tok, q_heads, hd)), dtype)
        self.n_pages = n_pages

    def device(self, ragged=True, interleave=False, err=True):
        """Device tensors; interleave: k and v pages side by side in one allocation."""
        dt = TYPES[self.dtype]
        if interleave:
            both = torch.empty((self.n_pages, 2) + self.k.shape[1:], dtype=dt, device="cuda")
            self.dk, self.dv = both[:, 0], both[:, 1]
            self.dk.copy_(to_dev(self.k, self.dtype))
            self.dv.copy_(to_dev(self.v, self.dtype))
        else:
            self.dk, self.dv = to_dev(self.k, self.dtype), to_dev(self.v, self.dtype)
        self.dtable = torch.from_numpy(self.table).cuda()
        self.dlen = torch.tensor(self.old, dtype=torch.int32, device="cuda")
        self.dcu = torch.from_numpy(self.cu).cuda() if ragged else None
        self.derr = torch.zeros(1, dtype=torch.int32, device="cuda") if err else None
        self.attn = binding.make_attn(
            q_heads=self.q_heads, k_pages=self.dk, v_pages=self.dv, page_table=self.dtable,
            kv_len=self.dlen, max_T=max(self.new + [0]), cu_seqlens=self.dcu, n_tok=self.n_tok,
            window=self.window, sinks=self.sinks, scale=self.scale, dev_err=self.derr)
        return self

    def run(self, q=None, lse=True, stream=None, workspace=None):
        q = to_dev(self.q, self.dtype) if q is None else q
        self.o = torch.full((self.n_tok, self.q_heads, self.hd), 7.0, dtype=TYPES[self.dtype],
                            device="cuda")
        self.lse = torch.full((self.n_tok, self.q_heads), 7.0, device="cuda") if lse else None
        self.ws = binding.paged_attn_workspace(self.attn) if workspace is None else workspace
        torch.cuda.synchronize()
        binding.gdn_paged_attn(self.attn, q, self.o, lse=self.lse, workspace=self.ws, stream=stream)
        torch.cuda.synchronize()
        return self

    def expected(self):
        return oracle.paged_attention(self.q, self.cu, self.old, self.k, self.v, self.table,
                                      self.scale, self.window, self.sinks)

    def check(self, rows=None):
        o, lse, mean = self.expected()
        rows = slice(None) if rows is None else rows
        check_close(self.o.float().cpu().numpy()[rows], o[rows], mean[rows], self.dtype)
        if self.lse is not None:
            # the scores' error, and that of a sum of some thousand float32 terms
            tol = (2.0 ** -12 if self.dtype == "bf16" else 2.0 ** -14) + 2.0 ** -20 * np.abs(lse[rows])
            assert np.all(np.abs(self.lse.cpu().numpy()[rows] - lse[rows]) <= tol)
        if self.derr is not None:
            assert int(self.derr.item()) == 0


def check_close(got, want, mean, dtype):
    tol = (2.0 ** -8 * (np.abs(want) + mean) + 2.0 ** -11 * mean if dtype == "bf16"
           else 2.0 ** -13 * mean) + 1e-30
    assert np.all(np.isfinite(got))
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), got.size, float(np.max(np.abs(got - want) / tol)))
