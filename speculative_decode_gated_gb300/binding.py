"""Python binding of libgdn.so: argument marshalling only.

Every function here has the name of the C entry point it calls (include/gdn.h)
and only turns torch tensors into device pointers and sizes; all computation
runs in the CUDA kernels.  If the library has not been built this module raises
on first use: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libgdn.so")

GDN_OK = 0
GDN_ERR_DEVICE_ARG = 5
GDN_ERR_ALIAS, GDN_ERR_LAYER_MISMATCH = 8, 9
GDN_FP32, GDN_BF16 = 0, 1
GDN_FLAG_O_BF16, GDN_FLAG_LOG_GATE = 1, 2
GDN_ALGO_AUTO, GDN_ALGO_RECURRENT, GDN_ALGO_CHUNK, GDN_ALGO_CHUNK_TC = 0, 1, 2, 3
GDN_DEVERR_SLOT, GDN_DEVERR_ACCEPTED, GDN_DEVERR_SEQLEN = 1, 2, 4
GDN_DEVERR_TIMEOUT, GDN_DEVERR_REPLAY = 8, 16
GDN_DEVERR_KV_LEN, GDN_DEVERR_PAGE = 32, 64
GDN_DEVERR_TOKEN, GDN_DEVERR_NO_PAGES = 128, 256
GDN_MAX_T = 1024
GDN_ATTN_MAX_T = 65536
GDN_MAX_VOCAB = 262144

# Every symbol include/gdn.h declares.
EXPORTED = (
    "gdn_verify", "gdn_commit", "gdn_verify_commit_fused",
    "gdn_verify_layers", "gdn_commit_layers", "gdn_verify_commit_fused_layers",
    "gdn_accept_prefix", "gdn_replay_verify", "gdn_replay_commit", "gdn_commit_verify",
    "gdn_read_device_error", "gdn_selftest_wait_timeout",
    "gdn_select_algo", "gdn_status_string", "gdn_last_error_string", "gdn_version",
    "gdn_rope_append", "gdn_paged_attn", "gdn_paged_attn_workspace", "gdn_read_attn_error",
    "gdn_linear_verify", "gdn_linear_commit", "gdn_linear_step", "gdn_accept_sample",
    "gdn_plan_pages", "gdn_read_error",
)


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {gdn_status_string(status)} (status {status})"
        if status == 6:
            msg += f": {gdn_last_error_string()}"
        super().__init__(msg)


class gdn_problem(ctypes.Structure):
    """Mirror of the C struct gdn_problem (include/gdn.h), field for field."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32), ("max_T", ctypes.c_int32), ("qkv_dtype", ctypes.c_int32),
        ("algo", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("cu_seqlens", ctypes.c_void_p), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("pool", ctypes.c_void_p), ("pool_slots", ctypes.c_int64),
        ("slot_ids", ctypes.c_void_p), ("dev_err", ctypes.c_void_p), ("n_tok", ctypes.c_int64),
    ]


class gdn_replay(ctypes.Structure):
    """Mirror of the C struct gdn_replay (include/gdn.h), field for field."""

    _fields_ = [
        ("capacity", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
        ("beta", ctypes.c_void_p), ("len_in", ctypes.c_void_p), ("len_out", ctypes.c_void_p),
    ]


class gdn_prev_step(ctypes.Structure):
    """Mirror of the C struct gdn_prev_step (include/gdn.h), field for field."""

    _fields_ = [
        ("cu_seqlens", ctypes.c_void_p), ("max_T", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("n_tok", ctypes.c_int64), ("k", ctypes.c_void_p), ("alpha", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("accepted", ctypes.c_void_p),
    ]


class gdn_attn(ctypes.Structure):
    """Mirror of the C struct gdn_attn (include/gdn.h), field for field."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("max_T", ctypes.c_int32), ("dtype", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
        ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p), ("n_tok", ctypes.c_int64),
        ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("n_pages", ctypes.c_int64),
        ("page_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p), ("dev_err", ctypes.c_void_p),
    ]


class gdn_rope(ctypes.Structure):
    """Mirror of the C struct gdn_rope (include/gdn.h), field for field."""

    _fields_ = [
        ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("mscale", ctypes.c_float),
        ("reserved", ctypes.c_int32), ("inv_freq", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


class gdn_linear(ctypes.Structure):
    """Mirror of the C struct gdn_linear (include/gdn.h), field for field."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("max_T", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("cu_seqlens", ctypes.c_void_p),
        ("n_tok", ctypes.c_int64), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("log_decay", ctypes.c_void_p),
        ("decay_stride", ctypes.c_int64), ("pool", ctypes.c_void_p), ("pool_slots", ctypes.c_int64),
        ("slot_ids", ctypes.c_void_p), ("dev_err", ctypes.c_void_p),
    ]


class gdn_sample(ctypes.Structure):
    """Mirror of the C struct gdn_sample (include/gdn.h), field for field."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("max_T", ctypes.c_int32), ("vocab", ctypes.c_int32),
        ("reserved", ctypes.c_int32), ("cu_seqlens", ctypes.c_void_p), ("n_tok", ctypes.c_int64),
        ("draft_ids", ctypes.c_void_p), ("target_probs", ctypes.c_void_p),
        ("target_stride", ctypes.c_int64), ("draft_probs", ctypes.c_void_p),
        ("draft_stride", ctypes.c_int64), ("u_accept", ctypes.c_void_p),
        ("u_sample", ctypes.c_void_p), ("dev_err", ctypes.c_void_p),
    ]


class gdn_pages(ctypes.Structure):
    """Mirror of the C struct gdn_pages (include/gdn.h), field for field."""

    _fields_ = [
        ("batch", ctypes.c_int32), ("max_T", ctypes.c_int32), ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("rows", ctypes.c_void_p),
        ("accepted", ctypes.c_void_p), ("done", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
        ("held", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("kv_len_out", ctypes.c_void_p),
        ("held_out", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p),
        ("free_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("max_rows", ctypes.c_int64), ("dev_err", ctypes.c_void_p),
    ]


_lib_handle: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it was never built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with speculative_decode_gated_gb300.build() "
                "(there is no CPU or PyTorch fallback)")
        h = ctypes.CDLL(LIB_PATH)
        P, S = ctypes.POINTER(gdn_problem), ctypes.c_void_p
        h.gdn_verify.argtypes = [P, S, S]
        h.gdn_commit.argtypes = [P, S, S]
        h.gdn_verify_commit_fused.argtypes = [P, S, S, S]
        I32 = ctypes.c_int32
        h.gdn_verify_layers.argtypes = [P, I32, S, S]
        h.gdn_commit_layers.argtypes = [P, I32, S, S]
        h.gdn_verify_commit_fused_layers.argtypes = [P, I32, S, S, S]
        h.gdn_accept_prefix.argtypes = [I32, I32, S, ctypes.c_int64, S, S, S, S, S]
        R = ctypes.POINTER(gdn_replay)
        h.gdn_replay_verify.argtypes = [P, R, S, S]
        h.gdn_replay_commit.argtypes = [P, R, S, S]
        h.gdn_commit_verify.argtypes = [P, ctypes.POINTER(gdn_prev_step), S, S, S]
        I64, A = ctypes.c_int64, ctypes.POINTER(gdn_attn)
        h.gdn_rope_append.argtypes = [A, ctypes.POINTER(gdn_rope), S, I64, S, I64, S, I64, S, S]
        h.gdn_paged_attn.argtypes = [A, S, I64, S, S, S, I64, S]
        h.gdn_paged_attn_workspace.argtypes = [A]
        h.gdn_paged_attn_workspace.restype = I64
        L = ctypes.POINTER(gdn_linear)
        h.gdn_linear_verify.argtypes = [L, S, S]
        h.gdn_linear_commit.argtypes = [L, S, S]
        h.gdn_linear_step.argtypes = [L, S, S]
        h.gdn_accept_sample.argtypes = [ctypes.POINTER(gdn_sample), S, S, S]
        h.gdn_plan_pages.argtypes = [ctypes.POINTER(gdn_pages), S]
        h.gdn_read_error.argtypes = [S, S, ctypes.POINTER(ctypes.c_int32)]
        h.gdn_read_device_error.argtypes = [P, S, ctypes.POINTER(ctypes.c_int32)]
        h.gdn_read_attn_error.argtypes = [A, S, ctypes.POINTER(ctypes.c_int32)]
        h.gdn_selftest_wait_timeout.argtypes = [S, S]
        h.gdn_select_algo.argtypes = [P]
        h.gdn_status_string.argtypes = [ctypes.c_int]
        for name in ("gdn_verify", "gdn_commit", "gdn_verify_commit_fused",
                     "gdn_verify_layers", "gdn_commit_layers", "gdn_verify_commit_fused_layers",
                     "gdn_accept_prefix", "gdn_replay_verify", "gdn_replay_commit",
                     "gdn_commit_verify", "gdn_read_device_error", "gdn_selftest_wait_timeout",
                     "gdn_select_algo", "gdn_rope_append", "gdn_paged_attn",
                     "gdn_read_attn_error", "gdn_linear_verify", "gdn_linear_commit",
                     "gdn_linear_step", "gdn_accept_sample", "gdn_plan_pages", "gdn_read_error"):
            getattr(h, name).restype = ctypes.c_int
        for name in ("gdn_status_string", "gdn_last_error_string", "gdn_version"):
            getattr(h, name).restype = ctypes.c_char_p
        _lib_handle = h
    return _lib_handle


class Problem:
    """A gdn_problem plus references to the tensors it points into."""

    def __init__(self, c: gdn_problem, refs: tuple):
        self.c = c
        self.refs = refs

    @property
    def ref(self):
        return ctypes.byref(self.c)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _check(t: Optional[torch.Tensor], name: str, dtypes, device) -> None:
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def make_problem(*, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                 beta: torch.Tensor, pool: torch.Tensor, slot_ids: torch.Tensor,
                 max_T: int, cu_seqlens: Optional[torch.Tensor] = None,
                 dev_err: Optional[torch.Tensor] = None, algo: int = GDN_ALGO_AUTO,
                 flags: int = 0) -> Problem:
    """Builds the C problem from device tensors (shapes as in include/gdn.h).

    q, k: [N_tok, H, dk]; v: [N_tok, H, dv] (bf16 or fp32, same dtype);
    alpha, beta: [N_tok, H] fp32; pool: [slots, H, dk, dv] fp32; slot_ids: [B] int32;
    cu_seqlens: [B+1] int32 or None (uniform length max_T); dev_err: [1] int32 or None.
    flags: GDN_FLAG_* bits (bf16 o, log-space alpha).  q may be None for a problem
    that only commits (the commit calls read no q).
    """
    dev = pool.device
    if k.dtype not in (torch.bfloat16, torch.float32) or v.dtype != k.dtype or \
            (q is not None and q.dtype != k.dtype):
        raise TypeError("q, k, v must all be bf16 or all fp32")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, (k.dtype,), dev)
    _check(alpha, "alpha", (torch.float32,), dev)
    _check(beta, "beta", (torch.float32,), dev)
    _check(pool, "pool", (torch.float32,), dev)
    _check(slot_ids, "slot_ids", (torch.int32,), dev)
    _check(cu_seqlens, "cu_seqlens", (torch.int32,), dev)
    _check(dev_err, "dev_err", (torch.int32,), dev)
    if pool.dim() != 4:
        raise ValueError("pool must be [slots, heads, dk, dv]")
    slots, H, dk, dv = pool.shape
    c = gdn_problem()
    c.batch = slot_ids.numel()
    c.heads, c.dk, c.dv = H, dk, dv
    c.max_T = int(max_T)
    c.qkv_dtype = GDN_BF16 if k.dtype == torch.bfloat16 else GDN_FP32
    c.algo = int(algo)
    c.flags = int(flags)
    c.cu_seqlens = _ptr(cu_seqlens)
    c.q, c.k, c.v = _ptr(q), _ptr(k), _ptr(v)
    c.alpha, c.beta = _ptr(alpha), _ptr(beta)
    c.pool = _ptr(pool)
    c.pool_slots = slots
    c.slot_ids = _ptr(slot_ids)
    c.dev_err = _ptr(dev_err)
    c.n_tok = k.shape[0]
    return Problem(c, (q, k, v, alpha, beta, pool, slot_ids, cu_seqlens, dev_err))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _raise(status: int, where: str) -> None:
    if status != GDN_OK:
        raise GdnError(status, where)


def _o_dtype(prob: Problem):
    return torch.bfloat16 if prob.c.flags & GDN_FLAG_O_BF16 else torch.float32


def gdn_verify(prob: Problem, o: torch.Tensor, stream=None) -> None:
    _check(o, "o", (_o_dtype(prob),), None)
    _raise(lib().gdn_verify(prob.ref, _ptr(o), _stream(stream)), "gdn_verify")


def gdn_commit(prob: Problem, accepted: torch.Tensor, stream=None) -> None:
    _check(accepted, "accepted", (torch.int32,), None)
    _raise(lib().gdn_commit(prob.ref, _ptr(accepted), _stream(stream)), "gdn_commit")


def gdn_verify_commit_fused(prob: Problem, accepted: torch.Tensor, o: torch.Tensor,
                            stream=None) -> None:
    _check(accepted, "accepted", (torch.int32,), None)
    _check(o, "o", (_o_dtype(prob),), None)
    _raise(lib().gdn_verify_commit_fused(prob.ref, _ptr(accepted), _ptr(o), _stream(stream)),
           "gdn_verify_commit_fused")


class ProblemArray:
    """A host array of gdn_problem (one per layer) for the layer-batch calls."""

    def __init__(self, problems):
        self.problems = list(problems)
        n = len(self.problems)
        self.c = (gdn_problem * max(n, 1))()
        for i, p in enumerate(self.problems):
            self.c[i] = p.c
        self.n = n

    @property
    def ref(self):
        return ctypes.cast(self.c, ctypes.POINTER(gdn_problem))


def _ptr_array(tensors) -> ctypes.Array:
    arr = (ctypes.c_void_p * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        _check(t, f"o[{i}]", (torch.float32, torch.bfloat16), None)
        arr[i] = _ptr(t)
    return arr


def gdn_verify_layers(probs: ProblemArray, o, stream=None) -> None:
    """o: one fp32 output tensor per layer."""
    arr = _ptr_array(o)
    _raise(lib().gdn_verify_layers(probs.ref, probs.n, arr, _stream(stream)), "gdn_verify_layers")


def gdn_commit_layers(probs: ProblemArray, accepted: torch.Tensor, stream=None) -> None:
    _check(accepted, "accepted", (torch.int32,), None)
    _raise(lib().gdn_commit_layers(probs.ref, probs.n, _ptr(accepted), _stream(stream)),
           "gdn_commit_layers")


def gdn_verify_commit_fused_layers(probs: ProblemArray, accepted: torch.Tensor, o,
                                   stream=None) -> None:
    _check(accepted, "accepted", (torch.int32,), None)
    arr = _ptr_array(o)
    _raise(lib().gdn_verify_commit_fused_layers(probs.ref, probs.n, _ptr(accepted), arr,
                                                _stream(stream)),
           "gdn_verify_commit_fused_layers")


def gdn_accept_prefix(draft_ids: torch.Tensor, target_ids: torch.Tensor, accepted: torch.Tensor,
                      max_T: int, cu_seqlens: Optional[torch.Tensor] = None,
                      dev_err: Optional[torch.Tensor] = None, stream=None) -> None:
    """accepted[r] <- greedy accepted length of request r (int32 tensors on one device;
    draft_ids/target_ids [N_tok], accepted [B], cu_seqlens [B+1] or None)."""
    dev = accepted.device
    for t, n in ((draft_ids, "draft_ids"), (target_ids, "target_ids"), (accepted, "accepted"),
                 (cu_seqlens, "cu_seqlens"), (dev_err, "dev_err")):
        _check(t, n, (torch.int32,), dev)
    batch = accepted.numel()
    st = lib().gdn_accept_prefix(batch, int(max_T), _ptr(cu_seqlens), draft_ids.numel(),
                                 _ptr(draft_ids), _ptr(target_ids), _ptr(accepted), _ptr(dev_err),
                                 _stream(stream))
    _raise(st, "gdn_accept_prefix")


def gdn_selftest_wait_timeout(dev_err: torch.Tensor, stream=None) -> None:
    """Runs the kernels' bounded wait on a barrier nothing completes: about two
    seconds later GDN_DEVERR_TIMEOUT is ORed into dev_err (int32, one element)."""
    _check(dev_err, "dev_err", (torch.int32,), dev_err.device)
    st = lib().gdn_selftest_wait_timeout(_ptr(dev_err), _stream(stream))
    _raise(st, "gdn_selftest_wait_timeout")


class Replay:
    """A gdn_replay plus references to the tensors it points into."""

    def __init__(self, c: gdn_replay, refs: tuple):
        self.c = c
        self.refs = refs

    @property
    def ref(self):
        return ctypes.byref(self.c)

    def swap_lengths(self) -> None:
        """len_in <-> len_out, for the next step."""
        self.c.len_in, self.c.len_out = self.c.len_out, self.c.len_in
        self.refs = self.refs[:4] + (self.refs[5], self.refs[4])


def make_replay(*, capacity: int, k: torch.Tensor, v: torch.Tensor, alpha: torch.Tensor,
                beta: torch.Tensor, len_in: torch.Tensor, len_out: torch.Tensor) -> Replay:
    """k: [slots*capacity, H, dk], v: [slots*capacity, H, dv] (the q/k/v dtype);
    alpha, beta: [slots*capacity, H] fp32; len_in, len_out: [slots] int32."""
    dev = len_in.device
    _check(k, "k", (torch.bfloat16, torch.float32), dev)
    _check(v, "v", (k.dtype,), dev)
    for t, n in ((alpha, "alpha"), (beta, "beta")):
        _check(t, n, (torch.float32,), dev)
    for t, n in ((len_in, "len_in"), (len_out, "len_out")):
        _check(t, n, (torch.int32,), dev)
    c = gdn_replay()
    c.capacity, c.reserved = int(capacity), 0
    c.k, c.v, c.alpha, c.beta = _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta)
    c.len_in, c.len_out = _ptr(len_in), _ptr(len_out)
    return Replay(c, (k, v, alpha, beta, len_in, len_out))


def gdn_replay_verify(prob: Problem, rb: Replay, o: torch.Tensor, stream=None) -> None:
    _check(o, "o", (_o_dtype(prob),), None)
    _raise(lib().gdn_replay_verify(prob.ref, rb.ref, _ptr(o), _stream(stream)), "gdn_replay_verify")


def gdn_replay_commit(prob: Problem, rb: Replay, accepted: torch.Tensor, stream=None) -> None:
    _check(accepted, "accepted", (torch.int32,), None)
    _raise(lib().gdn_replay_commit(prob.ref, rb.ref, _ptr(accepted), _stream(stream)),
           "gdn_replay_commit")


def gdn_read_device_error(prob: Problem, stream=None) -> int:
    """Synchronises the stream and returns the device error word (0 = none)."""
    code = ctypes.c_int32(0)
    st = lib().gdn_read_device_error(prob.ref, _stream(stream), ctypes.byref(code))
    if st not in (GDN_OK, GDN_ERR_DEVICE_ARG):
        _raise(st, "gdn_read_device_error")
    return int(code.value)


def gdn_select_algo(prob: Problem) -> int:
    return int(lib().gdn_select_algo(prob.ref))


def gdn_status_string(status: int) -> str:
    return lib().gdn_status_string(int(status)).decode()


def gdn_last_error_string() -> str:
    return lib().gdn_last_error_string().decode()


def gdn_version() -> str:
    return lib().gdn_version().decode()


class PrevStep:
    """A gdn_prev_step plus references to the tensors it points into."""

    def __init__(self, c: gdn_prev_step, refs: tuple):
        self.c = c
        self.refs = refs

    @property
    def ref(self):
        return ctypes.byref(self.c)


def make_prev_step(*, k: torch.Tensor, alpha: torch.Tensor, w: torch.Tensor,
                   accepted: torch.Tensor, max_T: int,
                   cu_seqlens: Optional[torch.Tensor] = None) -> PrevStep:
    """The previous step of the same requests: its k [N_tok, H, dk], alpha [N_tok, H],
    the w its gdn_commit_verify wrote [N_tok, H, dv] fp32, its accepted [B] int32,
    and its row offsets [B+1] int32 or None (uniform length max_T)."""
    dev = k.device
    _check(k, "k", (torch.bfloat16, torch.float32), dev)
    _check(alpha, "alpha", (torch.float32,), dev)
    _check(w, "w", (torch.float32,), dev)
    _check(accepted, "accepted", (torch.int32,), dev)
    _check(cu_seqlens, "cu_seqlens", (torch.int32,), dev)
    c = gdn_prev_step()
    c.cu_seqlens = _ptr(cu_seqlens)
    c.max_T, c.reserved = int(max_T), 0
    c.n_tok = k.shape[0]
    c.k, c.alpha, c.w, c.accepted = _ptr(k), _ptr(alpha), _ptr(w), _ptr(accepted)
    return PrevStep(c, (k, alpha, w, accepted, cu_seqlens))


def gdn_commit_verify(prob: Problem, prev: Optional[PrevStep], o: torch.Tensor, w: torch.Tensor,
                      stream=None) -> None:
    """Commit `prev` (None: nothing), then verify `prob`; w: this step's W [N_tok, H, dv] fp32."""
    _check(o, "o", (_o_dtype(prob),), None)
    _check(w, "w", (torch.float32,), None)
    _raise(lib().gdn_commit_verify(prob.ref, None if prev is None else prev.ref, _ptr(o), _ptr(w),
                                   _stream(stream)), "gdn_commit_verify")


class Attn:
    """A gdn_attn (the requests, their paged cache and the mask of one attention layer)
    plus references to the tensors it points into."""

    def __init__(self, c: gdn_attn, refs: tuple, dtype, device):
        self.c = c
        self.refs = refs
        self.dtype, self.device = dtype, device
        self.index = device.index if device.type == "cuda" else None
        self.n_tok, self.q_heads, self.kv_heads, self.head_dim = (
            c.n_tok, c.q_heads, c.kv_heads, c.head_dim)
        self.ref = ctypes.byref(c)


def make_attn(*, q_heads: int, k_pages: torch.Tensor, v_pages: torch.Tensor,
              page_table: torch.Tensor, kv_len: torch.Tensor, max_T: int,
              cu_seqlens: Optional[torch.Tensor] = None, n_tok: Optional[int] = None,
              window: int = 0, sinks: int = 0, scale: Optional[float] = None,
              dev_err: Optional[torch.Tensor] = None) -> Attn:
    """Builds the C description of one attention layer's step (include/gdn.h).

    k_pages, v_pages: [n_pages, kv_heads, page_size, head_dim] bf16 or fp32, each page
    contiguous, pages any equal distance apart; page_table: [B, max_pages] int32;
    kv_len: [B] int32, the tokens cached before the step; cu_seqlens: [B+1] int32 with
    n_tok rows, or None (uniform length max_T).  window: 0, or the last places a row
    sees; sinks: first places that stay visible under it.  scale: 1 / sqrt(head_dim)
    when None."""
    dev = k_pages.device
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("k_pages and v_pages must both be [n_pages, kv_heads, page_size, head_dim]")
    if k_pages.dtype not in (torch.bfloat16, torch.float32) or v_pages.dtype != k_pages.dtype:
        raise TypeError("k_pages and v_pages must both be bf16 or both fp32")
    n_pages, kv_heads, page, hd = k_pages.shape
    for t, n in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")
        # (the distance of a single head's rows from the next head's has no meaning)
        if t.stride()[2:] != (hd, 1) or (t.stride(1) != page * hd and kv_heads > 1):
            raise ValueError(f"a page of {n} must be contiguous")
    if n_pages > 1 and v_pages.stride(0) != k_pages.stride(0):
        raise ValueError("k_pages and v_pages must have the same page stride")
    for t, n in ((page_table, "page_table"), (kv_len, "kv_len"), (cu_seqlens, "cu_seqlens"),
                 (dev_err, "dev_err")):
        _check(t, n, (torch.int32,), dev)
    batch = kv_len.numel()
    if page_table.dim() != 2 or page_table.shape[0] != batch:
        raise ValueError("page_table must be [batch, max_pages]")
    if cu_seqlens is not None and (cu_seqlens.numel() != batch + 1 or n_tok is None):
        raise ValueError("a ragged step needs cu_seqlens [batch + 1] and n_tok")
    c = gdn_attn()
    c.batch, c.q_heads, c.kv_heads, c.head_dim = batch, int(q_heads), kv_heads, hd
    c.max_T = int(max_T)
    c.dtype = GDN_BF16 if k_pages.dtype == torch.bfloat16 else GDN_FP32
    c.page_size, c.max_pages = page, page_table.shape[1]
    c.window, c.sinks = int(window), int(sinks)
    c.scale = hd ** -0.5 if scale is None else float(scale)
    c.cu_seqlens = _ptr(cu_seqlens)
    c.n_tok = int(n_tok) if cu_seqlens is not None else batch * int(max_T)
    c.k_pages, c.v_pages = _ptr(k_pages), _ptr(v_pages)
    c.n_pages = n_pages
    c.page_stride = k_pages.stride(0) if n_pages > 1 else kv_heads * page * hd
    c.page_table, c.kv_len, c.dev_err = _ptr(page_table), _ptr(kv_len), _ptr(dev_err)
    return Attn(c, (k_pages, v_pages, page_table, kv_len, cu_seqlens, dev_err), k_pages.dtype, dev)


class Rope:
    """A gdn_rope plus references to the tensors it points into."""

    def __init__(self, c: gdn_rope, refs: tuple):
        self.c = c
        self.refs = refs
        self.ref = ctypes.byref(c)


def make_rope(*, inv_freq: torch.Tensor, interleaved: bool = False, mscale: float = 1.0,
              positions: Optional[torch.Tensor] = None) -> Rope:
    """inv_freq: [rot_dim / 2] fp32, radians per position (staging.rope_frequencies);
    positions: [N_tok] int32, or None (a row's position is its place in the cache)."""
    _check(inv_freq, "inv_freq", (torch.float32,), None)
    _check(positions, "positions", (torch.int32,), inv_freq.device)
    c = gdn_rope()
    c.rot_dim, c.interleaved = 2 * inv_freq.numel(), int(bool(interleaved))
    c.mscale, c.reserved = float(mscale), 0
    c.inv_freq, c.positions = _ptr(inv_freq), _ptr(positions)
    return Rope(c, (inv_freq, positions))


def _check_rows(t: torch.Tensor, name: str, attn: Attn, heads: int) -> int:
    """Checks a [N_tok, heads, head_dim] tensor whose rows are contiguous; its row stride."""
    n, hd = attn.n_tok, attn.head_dim
    if t.dtype is not attn.dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {attn.dtype}")
    if t.device != attn.device:
        raise ValueError(f"{name} is on {t.device}, expected {attn.device}")
    if t.shape != (n, heads, hd):
        raise ValueError(f"{name} must be {(n, heads, hd)}, is {tuple(t.shape)}")
    s = t.stride()
    if s[2] != 1 or (s[1] != hd and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return s[0] if n > 1 else heads * hd


def _elsewhere(attn: Attn) -> bool:
    """Whether another device than the tensors' is current, where the kernels would go."""
    return attn.index is not None and torch._C._cuda_getDevice() != attn.index


def _attn_stream(attn: Attn, stream) -> int:
    """`stream`, or the current stream of the tensors' device, which is the current device."""
    if attn.index is None:
        raise ValueError(f"the tensors are on {attn.device}, expected a CUDA device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(attn.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def gdn_rope_append(attn: Attn, rope: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                    q_out: torch.Tensor, stream=None) -> None:
    """q_out <- rotated q; the rotated k and the v of each row to the pages.
    q, q_out: [N_tok, q_heads, head_dim]; k, v: [N_tok, kv_heads, head_dim]; the rows of
    q, k and v may be slices of wider ones, q_out is contiguous."""
    if _elsewhere(attn):
        with torch.cuda.device(attn.index):
            return gdn_rope_append(attn, rope, q, k, v, q_out, stream)
    Hq, Hkv = attn.q_heads, attn.kv_heads
    sq, sk = _check_rows(q, "q", attn, Hq), _check_rows(k, "k", attn, Hkv)
    sv = _check_rows(v, "v", attn, Hkv)
    if _check_rows(q_out, "q_out", attn, Hq) != Hq * attn.head_dim:
        raise ValueError("q_out must be contiguous")
    inv_freq, positions = rope.refs
    if inv_freq.device != attn.device:
        raise ValueError(f"inv_freq is on {inv_freq.device}, expected {attn.device}")
    if positions is not None and positions.numel() != attn.n_tok:
        raise ValueError("positions must be [N_tok]")
    st = lib().gdn_rope_append(attn.ref, rope.ref, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(),
                               sv, q_out.data_ptr(), _attn_stream(attn, stream))
    if st:
        _raise(st, "gdn_rope_append")


def gdn_paged_attn_workspace(attn: Attn) -> int:
    """Bytes of workspace that gdn_paged_attn needs."""
    n = int(lib().gdn_paged_attn_workspace(attn.ref))
    if n < 0:
        raise ValueError("gdn_paged_attn_workspace: the sizes are not valid")
    return n


def paged_attn_workspace(attn: Attn) -> torch.Tensor:
    """A workspace for gdn_paged_attn, zero-filled (on the current stream); one per stream, kept
    from call to call."""
    return torch.zeros(gdn_paged_attn_workspace(attn), dtype=torch.uint8, device=attn.device)


def gdn_paged_attn(attn: Attn, q: torch.Tensor, o: torch.Tensor, *, workspace: torch.Tensor,
                   lse: Optional[torch.Tensor] = None, stream=None) -> None:
    """o <- attention of the step's rows over the cache; lse (fp32 [N_tok, q_heads], or None)
    <- the logarithm of each row's sum.  q, o: [N_tok, q_heads, head_dim]; q's rows may be
    slices of wider ones, o is contiguous."""
    if _elsewhere(attn):
        with torch.cuda.device(attn.index):
            return gdn_paged_attn(attn, q, o, workspace=workspace, lse=lse, stream=stream)
    Hq = attn.q_heads
    sq = _check_rows(q, "q", attn, Hq)
    if _check_rows(o, "o", attn, Hq) != Hq * attn.head_dim:
        raise ValueError("o must be contiguous")
    if lse is not None:
        _check(lse, "lse", (torch.float32,), attn.device)
        if lse.numel() != attn.n_tok * Hq:
            raise ValueError("lse must be [N_tok, q_heads]")
    if workspace.device != attn.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {attn.device}")
    st = lib().gdn_paged_attn(attn.ref, q.data_ptr(), sq, o.data_ptr(), _ptr(lse),
                              workspace.data_ptr(), workspace.nbytes, _attn_stream(attn, stream))
    if st:
        _raise(st, "gdn_paged_attn")


def gdn_read_attn_error(attn: Attn, stream=None) -> int:
    """Waits for the stream and returns the error word of `attn` (GDN_DEVERR_* bits, 0: none)."""
    if _elsewhere(attn):
        with torch.cuda.device(attn.index):
            return gdn_read_attn_error(attn, stream)
    code = ctypes.c_int32(0)
    st = lib().gdn_read_attn_error(attn.ref, _attn_stream(attn, stream), ctypes.byref(code))
    if st not in (GDN_OK, GDN_ERR_DEVICE_ARG):
        _raise(st, "gdn_read_attn_error")
    return code.value


# ------------------------------------------------------------------ linear attention

class _Call:
    """A C struct plus the tensors it points into and the device that the call runs on."""

    def __init__(self, c, refs: tuple, device):
        self.c = c
        self.refs = refs
        self.device = device
        self.index = device.index if device.type == "cuda" else None
        self.ref = ctypes.byref(c)


class Linear(_Call):
    """A gdn_linear (one linear attention layer's step)."""

    def __init__(self, c: gdn_linear, refs: tuple, dtype, device):
        super().__init__(c, refs, device)
        self.dtype = dtype
        self.o_shape = (c.n_tok, c.heads, c.dv)
        self.batch = c.batch


def _same_device(t: Optional[torch.Tensor], name: str, device) -> None:
    if t is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _heads_rows(t: torch.Tensor, name: str, n: int, heads: int, dim: int) -> int:
    """Checks that t is [n, heads, dim] with the heads of a row contiguous; its row stride."""
    if t.dim() != 3 or t.shape != (n, heads, dim):
        raise ValueError(f"{name} must be {(n, heads, dim)}, is {tuple(t.shape)}")
    if n == 0:
        return heads * dim
    s = t.stride()
    if s[2] != 1 or (s[1] != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return s[0] if n > 1 else heads * dim


def make_linear(*, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                pool: torch.Tensor, slot_ids: torch.Tensor, max_T: int,
                cu_seqlens: Optional[torch.Tensor] = None, scale: float = 1.0,
                dev_err: Optional[torch.Tensor] = None) -> Linear:
    """Builds the C description of one linear attention layer's step (include/gdn.h).

    q, k: [N_tok, k_heads, dk], v: [N_tok, heads, dv], all bf16 or all fp32, rows any equal distance
    apart (slices of a projection's output); q may be None for gdn_linear_commit.  log_decay:
    fp32, [heads] (constants) or [N_tok, heads]; pool: [slots, heads, dk, dv] fp32; slot_ids: [B]
    int32; cu_seqlens: [B+1] int32 or None (uniform length max_T)."""
    dev = pool.device
    if pool.dim() != 4:
        raise ValueError("pool must be [slots, heads, dk, dv]")
    slots, H, dk, dv = pool.shape
    if k.dtype not in (torch.bfloat16, torch.float32) or v.dtype != k.dtype or \
            (q is not None and q.dtype != k.dtype):
        raise TypeError("q, k, v must all be bf16 or all fp32")
    _check(pool, "pool", (torch.float32,), dev)
    _check(slot_ids, "slot_ids", (torch.int32,), dev)
    _check(cu_seqlens, "cu_seqlens", (torch.int32,), dev)
    _check(dev_err, "dev_err", (torch.int32,), dev)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (log_decay, "log_decay")):
        _same_device(t, n, dev)
    batch = slot_ids.numel()
    if cu_seqlens is not None and cu_seqlens.numel() != batch + 1:
        raise ValueError("cu_seqlens must be [batch + 1]")
    if k.dim() != 3:
        raise ValueError("k must be [N_tok, k_heads, dk]")
    n = k.shape[0]
    if cu_seqlens is None and n != batch * int(max_T):
        raise ValueError(f"a uniform step has batch * max_T = {batch * int(max_T)} rows, k has {n}")
    Hk = k.shape[1]
    c = gdn_linear()
    c.batch, c.heads, c.k_heads, c.dk, c.dv, c.max_T = batch, H, Hk, dk, dv, int(max_T)
    c.dtype = GDN_BF16 if k.dtype == torch.bfloat16 else GDN_FP32
    c.scale = float(scale)
    c.cu_seqlens, c.n_tok = _ptr(cu_seqlens), n
    c.k_stride, c.v_stride = _heads_rows(k, "k", n, Hk, dk), _heads_rows(v, "v", n, H, dv)
    c.q_stride = c.k_stride if q is None else _heads_rows(q, "q", n, Hk, dk)
    c.q, c.k, c.v = _ptr(q), _ptr(k), _ptr(v)
    if log_decay.dtype != torch.float32:
        raise TypeError(f"log_decay: dtype {log_decay.dtype}, expected torch.float32")
    if log_decay.shape == (H,):
        if not log_decay.is_contiguous():
            raise ValueError("log_decay must be contiguous")
        c.decay_stride = 0
    elif log_decay.shape == (n, H):
        if log_decay.stride(1) != 1 and H > 1:
            raise ValueError("log_decay: the heads of a row must be contiguous")
        # (one row, or rows that an expand() made the same: constants)
        c.decay_stride = log_decay.stride(0) if n > 1 else 0
    else:
        raise ValueError(f"log_decay must be {(H,)} or {(n, H)}, is {tuple(log_decay.shape)}")
    c.log_decay = _ptr(log_decay)
    c.pool, c.pool_slots, c.slot_ids, c.dev_err = _ptr(pool), slots, _ptr(slot_ids), _ptr(dev_err)
    return Linear(c, (q, k, v, log_decay, pool, slot_ids, cu_seqlens, dev_err), k.dtype, dev)


def _call(fn, name: str, call: _Call, stream, *args) -> None:
    """fn(struct, *args, stream) on the call's own device."""
    index = call.index
    if index is None:
        raise ValueError(f"the tensors are on {call.device}, expected a CUDA device")
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(fn, name, call, stream, *args)
    st = fn(call.ref, *args, _attn_stream(call, stream))
    if st:
        _raise(st, name)


def _check_o(lin: Linear, o: torch.Tensor) -> None:
    if o.dtype is not lin.dtype:
        raise TypeError(f"o: dtype {o.dtype}, expected {lin.dtype}")
    if o.device != lin.device:
        raise ValueError(f"o is on {o.device}, expected {lin.device}")
    if o.shape != lin.o_shape or not o.is_contiguous():
        raise ValueError(f"o must be contiguous and {lin.o_shape}, is {tuple(o.shape)}")


def _check_requests(t: torch.Tensor, name: str, call: _Call, batch: int) -> None:
    _check(t, name, (torch.int32,), call.device)
    if t.numel() != batch:
        raise ValueError(f"{name} must be [batch] = [{batch}]")


def gdn_linear_verify(lin: Linear, o: torch.Tensor, stream=None) -> None:
    """o [N_tok, heads, dv] (the type of q) for every row; the states stay."""
    _check_o(lin, o)
    _call(lib().gdn_linear_verify, "gdn_linear_verify", lin, stream, o.data_ptr())


def gdn_linear_commit(lin: Linear, accepted: torch.Tensor, stream=None) -> None:
    """The states after the first accepted[r] rows (int32 [batch]) into the pool."""
    _check_requests(accepted, "accepted", lin, lin.batch)
    _call(lib().gdn_linear_commit, "gdn_linear_commit", lin, stream, accepted.data_ptr())


def gdn_linear_step(lin: Linear, o: torch.Tensor, stream=None) -> None:
    """o for every row, and the states after the last one into the pool."""
    _check_o(lin, o)
    _call(lib().gdn_linear_step, "gdn_linear_step", lin, stream, o.data_ptr())


# ------------------------------------------------------------------ sampled drafts

class Sample(_Call):
    """A gdn_sample (drafts, both models' probabilities and the random numbers of a step)."""

    def __init__(self, c: gdn_sample, refs: tuple, device):
        super().__init__(c, refs, device)
        self.batch = c.batch


def _probs(t: torch.Tensor, name: str, n: int, vocab: int, device) -> int:
    if t.dtype != torch.float32:
        raise TypeError(f"{name}: dtype {t.dtype}, expected torch.float32")
    _same_device(t, name, device)
    if t.dim() != 2 or t.shape != (n, vocab):
        raise ValueError(f"{name} must be {(n, vocab)}, is {tuple(t.shape)}")
    if n and vocab > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a row must be contiguous")
    return t.stride(0) if n > 1 else vocab


def make_sample(*, draft_ids: torch.Tensor, target_probs: torch.Tensor, u_accept: torch.Tensor,
                u_sample: torch.Tensor, max_T: int, draft_probs: Optional[torch.Tensor] = None,
                cu_seqlens: Optional[torch.Tensor] = None,
                dev_err: Optional[torch.Tensor] = None) -> Sample:
    """Builds the C description of one acceptance (include/gdn.h).

    draft_ids: [N_tok] int32, the step's rows (each request's last token, then its drafts);
    target_probs, draft_probs: [N_tok, vocab] fp32, rows any equal distance apart; draft_probs None:
    drafts without a distribution; u_accept: [N_tok], u_sample: [B] fp32 in [0, 1); cu_seqlens:
    [B+1] int32 or None (uniform length max_T)."""
    dev = u_sample.device
    for t, n in ((draft_ids, "draft_ids"), (cu_seqlens, "cu_seqlens"), (dev_err, "dev_err")):
        _check(t, n, (torch.int32,), dev)
    for t, n in ((u_accept, "u_accept"), (u_sample, "u_sample")):
        _check(t, n, (torch.float32,), dev)
    batch, n = u_sample.numel(), draft_ids.numel()
    if cu_seqlens is not None and cu_seqlens.numel() != batch + 1:
        raise ValueError("cu_seqlens must be [batch + 1]")
    if cu_seqlens is None and n != batch * int(max_T):
        raise ValueError(f"a uniform step has batch * max_T = {batch * int(max_T)} rows, draft_ids has {n}")
    if u_accept.numel() != n:
        raise ValueError("u_accept must be [N_tok]")
    if target_probs.dim() != 2:
        raise ValueError("target_probs must be [N_tok, vocab]")
    c = gdn_sample()
    c.batch, c.max_T, c.vocab, c.reserved = batch, int(max_T), target_probs.shape[1], 0
    c.cu_seqlens, c.n_tok, c.draft_ids = _ptr(cu_seqlens), n, _ptr(draft_ids)
    c.target_stride = _probs(target_probs, "target_probs", n, c.vocab, dev)
    c.target_probs, c.draft_probs = _ptr(target_probs), _ptr(draft_probs)
    c.draft_stride = c.vocab if draft_probs is None else _probs(draft_probs, "draft_probs", n, c.vocab, dev)
    c.u_accept, c.u_sample, c.dev_err = _ptr(u_accept), _ptr(u_sample), _ptr(dev_err)
    return Sample(c, (draft_ids, target_probs, draft_probs, u_accept, u_sample, cu_seqlens, dev_err), dev)


def gdn_accept_sample(sample: Sample, accepted: torch.Tensor, next_ids: torch.Tensor,
                      stream=None) -> None:
    """accepted [B] <- rows kept of each request (what the commit calls take), next_ids [B] <- the
    token that follows them (int32)."""
    _check_requests(accepted, "accepted", sample, sample.batch)
    _check_requests(next_ids, "next_ids", sample, sample.batch)
    _call(lib().gdn_accept_sample, "gdn_accept_sample", sample, stream, accepted.data_ptr(),
          next_ids.data_ptr())


# ------------------------------------------------------------------ pages

class Pages(_Call):
    """A gdn_pages (the lengths, page table and free list of a paged cache)."""


def make_pages(*, page_table: torch.Tensor, page_size: int, max_T: int, kv_len: torch.Tensor,
               held: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
               cu_seqlens: torch.Tensor, rows: Optional[torch.Tensor] = None,
               accepted: Optional[torch.Tensor] = None, done: Optional[torch.Tensor] = None,
               kv_len_out: Optional[torch.Tensor] = None, held_out: Optional[torch.Tensor] = None,
               free_count_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None,
               dev_err: Optional[torch.Tensor] = None) -> Pages:
    """Builds the C description of a paged cache's next step (include/gdn.h).

    int32 tensors: page_table [B, max_pages], kv_len and held [B], free_pages [n_pages], free_count
    [1], cu_seqlens [B+1] (written), rows, accepted and done [B] or None; kv_len_out, held_out and
    free_count_out: None for in place.  slots (int64) and positions (int32) [max_rows], written, or
    None."""
    dev = page_table.device
    if page_table.dim() != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    batch, max_pages = page_table.shape
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    held_out = held if held_out is None else held_out
    free_count_out = free_count if free_count_out is None else free_count_out
    for t, n, size in ((page_table, "page_table", None), (kv_len, "kv_len", batch), (held, "held", batch),
                       (rows, "rows", batch), (accepted, "accepted", batch), (done, "done", batch),
                       (kv_len_out, "kv_len_out", batch), (held_out, "held_out", batch),
                       (free_count, "free_count", 1), (free_count_out, "free_count_out", 1),
                       (cu_seqlens, "cu_seqlens", batch + 1), (free_pages, "free_pages", None),
                       (positions, "positions", None), (dev_err, "dev_err", None)):
        _check(t, n, (torch.int32,), dev)
        if t is not None and size is not None and t.numel() != size:
            raise ValueError(f"{n} must have {size} entries, has {t.numel()}")
    _check(slots, "slots", (torch.int64,), dev)
    sizes = {t.numel() for t in (slots, positions) if t is not None}
    if len(sizes) > 1:
        raise ValueError("slots and positions must have the same size")
    c = gdn_pages()
    c.batch, c.max_T, c.page_size, c.max_pages = batch, int(max_T), int(page_size), max_pages
    c.n_pages = free_pages.numel()
    c.rows, c.accepted, c.done = _ptr(rows), _ptr(accepted), _ptr(done)
    c.kv_len, c.held, c.free_count = _ptr(kv_len), _ptr(held), _ptr(free_count)
    c.kv_len_out, c.held_out, c.free_count_out = _ptr(kv_len_out), _ptr(held_out), _ptr(free_count_out)
    c.free_pages, c.page_table, c.cu_seqlens = _ptr(free_pages), _ptr(page_table), _ptr(cu_seqlens)
    c.slots, c.positions = _ptr(slots), _ptr(positions)
    c.max_rows = sizes.pop() if sizes else 0
    c.dev_err = _ptr(dev_err)
    return Pages(c, (page_table, kv_len, held, free_pages, free_count, cu_seqlens, rows, accepted, done,
                     kv_len_out, held_out, free_count_out, slots, positions, dev_err), dev)


def gdn_plan_pages(pages: Pages, stream=None) -> None:
    """The next step's lengths, pages, row offsets, slots and positions."""
    _call(lib().gdn_plan_pages, "gdn_plan_pages", pages, stream)


def gdn_read_error(dev_err: torch.Tensor, stream=None) -> int:
    """Waits for the stream and returns an error word (GDN_DEVERR_* bits, 0: none)."""
    _check(dev_err, "dev_err", (torch.int32,), None)
    if dev_err.device.type != "cuda":
        raise ValueError(f"dev_err is on {dev_err.device}, expected a CUDA device")
    code = ctypes.c_int32(0)
    with torch.cuda.device(dev_err.device):
        st = lib().gdn_read_error(_ptr(dev_err), _stream(stream), ctypes.byref(code))
    if st not in (GDN_OK, GDN_ERR_DEVICE_ARG):
        _raise(st, "gdn_read_error")
    return code.value
