/*
 * gdn.h - C ABI of the Gated DeltaNet speculative verify/commit library (libgdn.so).
 *
 * The operation.  Gated DeltaNet (GDN) layers keep a fixed-size recurrent state
 * per request and head, read and rewritten for every token; ReplaySSM keeps a
 * checkpoint of that state, computes the draft tokens' outputs from the
 * checkpoint and the buffered inputs, and on rejection keeps only the accepted
 * prefix (OCRia write-up "OCRia 推理栈：单卡 B200 提速近 10 倍", section "Make
 * speculative verification cheaper"; the same in "Wie OCRia einen 10-fachen
 * Inference-Speedup auf B200-GPUs erreichte", section "Wie es funktioniert").  The state
 * update is the gated delta rule, with S the dv x dk state of one unit
 * (request r, head h):
 *
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T
 *     o_t = S_t q_t
 *
 * Layout (all row-major, all device memory, all caller-owned):
 *   state tile  float32 [dk][dv], tile[i][j] = S[j][i] (key index i is the row,
 *               value index j contiguous); 64 KiB at dk = dv = 128.
 *   pool        float32 [pool_slots][heads][dk][dv]; request r's checkpoint is
 *               pool[slot_ids[r]][h].
 *   q, k        [N_tok][heads][dk], v [N_tok][heads][dv], bfloat16 or float32
 *               (qkv_dtype); token rows of request r are [cu[r], cu[r+1]) with
 *               cu = cu_seqlens, or [r*max_T, (r+1)*max_T) when cu_seqlens is NULL.
 *   alpha, beta float32 [N_tok][heads] (alpha is the decay gate, beta the write
 *               strength; both given directly, no activation applied; with
 *               GDN_FLAG_LOG_GATE alpha holds g and the decay is expf(g)).
 *   o           float32 [N_tok][heads][dv] (bfloat16 with GDN_FLAG_O_BF16).
 *   accepted    int32 [batch], a_r in [0, T_r].
 *
 * Calls.  All compute calls are asynchronous on `stream`; they validate their
 * arguments on the host first and return an error without launching anything
 * if a check fails.  They allocate no memory and keep no state between calls.
 *   gdn_verify               o_t for every draft token; never writes the pool.
 *   gdn_commit               pool[slot_r][h] <- state after a_r tokens, for
 *                            every r with a_r > 0; slots with a_r = 0 and slots
 *                            no request names are left bit-identical.
 *   gdn_verify_commit_fused  both in one pass: reads each checkpoint once,
 *                            writes o for every token and the state once.
 *   gdn_commit_verify        the previous step's commit, then this step's
 *                            verify, in one pass (the order an engine can run
 *                            them in: a step's accepted lengths are known only
 *                            after all its layers verified).
 *   gdn_*_layers             the same calls for the layers of one step, in as
 *                            few launches as possible.
 *   gdn_replay_verify/commit a multi-step ReplaySSM buffer: outputs from the
 *                            checkpoint plus buffered rows, periodic flush.
 *   gdn_accept_prefix        greedy accepted lengths from token ids, on the
 *                            device.
 *   gdn_rope_append          attention layers: rotary positions of a step's
 *                            queries and keys, keys and values written to the
 *                            pages of a key/value cache.
 *   gdn_paged_attn           attention of the step's rows over that cache, all
 *                            of it or a sliding window with first tokens that
 *                            stay visible.
 *   gdn_read_attn_error      the device error word of an attention layer's step.
 *   gdn_linear_verify/commit/step  linear attention with a decay for each head over
 *                            the same kind of state pool: drafts and their accepted
 *                            prefix, single tokens and prompts.
 *   gdn_accept_sample        accepted lengths and next tokens of drafts that were
 *                            sampled, from both models' probabilities and given
 *                            random numbers, on the device.
 *   gdn_plan_pages           the next step's cache lengths, page table, row offsets,
 *                            slots and positions, from lengths on the device.
 *   gdn_read_error           any device error word.
 *   gdn_selftest_wait_timeout  runs the bounded wait to its expiry (diagnostic).
 *
 * Device-side argument errors (a slot id outside [0, pool_slots), a_r outside
 * [0, T_r], a ragged length outside [0, max_T]) cannot be seen on the host
 * without a synchronisation; the kernel ORs a GDN_DEVERR_* bit into *dev_err
 * (when dev_err is not NULL) and skips that unit, writing nothing for it.  It
 * never traps.  The chunked kernel's internal waits give up after about two
 * seconds and report GDN_DEVERR_TIMEOUT instead of hanging.  Duplicate slot
 * ids among the requests of one call are a precondition violation: commit
 * results are then undefined.
 */
#ifndef GDN_H
#define GDN_H

#include <stdint.h>

#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_NULL_PTR = 1,     /* a required pointer is NULL */
    GDN_ERR_BAD_DIM = 2,      /* batch/heads/max_T/pool_slots/n_tok out of range (token rows,
                                 batch*max_T or n_tok, above 2^31 - 1), or unknown flags */
    GDN_ERR_BAD_DTYPE = 3,    /* qkv_dtype is not a gdn_dtype */
    GDN_ERR_UNSUPPORTED = 4,  /* dk/dv (or a forced algo) not supported */
    GDN_ERR_DEVICE_ARG = 5,   /* reported by gdn_read_device_error, gdn_read_attn_error and gdn_read_error only */
    GDN_ERR_CUDA = 6,         /* a CUDA call failed; see gdn_last_error_string */
    GDN_ERR_ALIGN = 7,        /* a pointer is not aligned (16 bytes for q/k/v/pool/o) */
    GDN_ERR_ALIAS = 8,        /* o overlaps an input, or the pool overlaps q/k/v/o */
    GDN_ERR_LAYER_MISMATCH = 9 /* the problems of a layer batch disagree on a shared field */
} gdn_status;

typedef enum gdn_dtype {
    GDN_FP32 = 0,
    GDN_BF16 = 1
} gdn_dtype;

/* Which kernel runs.  AUTO: the chunked tensor-core kernel where it applies
 * (bf16 q/k/v, dk = dv = 128, any max_T: blocks of 16 tokens chained through
 * the state), else the recurrent kernel. */
typedef enum gdn_algo {
    GDN_ALGO_AUTO = 0,
    GDN_ALGO_RECURRENT = 1,   /* per-token update on CUDA cores, any supported shape */
    GDN_ALGO_CHUNK = 2,       /* WY/chunk form, bf16 mma.sync for the state products; 16-token
                                 chunks, the state carried from one chunk to the next */
    GDN_ALGO_CHUNK_TC = 3     /* the same chunk form with the two state-sized products on
                                 tcgen05.mma (A = H^T staged in tensor memory, accumulators in
                                 tensor memory) and the small solves on CUDA cores; same shapes
                                 as GDN_ALGO_CHUNK, results within the same tolerance; opt-in
                                 (slower than GDN_ALGO_CHUNK on 16-token chunks); no replay
                                 buffer calls; layer batches run one launch per layer */
} gdn_algo;

/* Bits ORed into *dev_err by the kernels. */
#define GDN_DEVERR_SLOT     1   /* slot_ids[r] outside [0, pool_slots) */
#define GDN_DEVERR_ACCEPTED 2   /* accepted[r] outside [0, T_r]        */
#define GDN_DEVERR_SEQLEN   4   /* cu[r+1] - cu[r] outside [0, max_T], or rows outside [0, n_tok) */
#define GDN_DEVERR_TIMEOUT  8   /* an internal pipeline wait gave up (about 2 s); results incomplete.
                                   The block that gave up also bounds its wait for its own
                                   copies in flight; if that wait gives up too, copies (or, on
                                   the tcgen05 kernel, products) may still land after the kernel
                                   ends.  Treat every later result on the stream as suspect until
                                   the CUDA context has been rebuilt. */
#define GDN_DEVERR_REPLAY  16   /* replay buffer: len_in[slot] < 0, or buffered plus new rows > capacity */
#define GDN_DEVERR_KV_LEN  32   /* cache: kv_len[r] < 0, or kv_len[r] + T_r > max_pages * page_size */
#define GDN_DEVERR_PAGE    64   /* cache: a page id that the call needs is outside [0, n_pages);
                                   gdn_plan_pages: the free list's count is */
#define GDN_DEVERR_TOKEN  128   /* a draft id outside [0, vocab), or a row without any probability */
#define GDN_DEVERR_NO_PAGES 256 /* the free list has too few pages for a request's next rows */

/* Variant bits of gdn_problem.flags (the same in every problem of a layer batch). */
#define GDN_FLAG_O_BF16    1    /* o is bfloat16 [N_tok][heads][dv], round to nearest even of the
                                   float32 result; otherwise o is float32 */
#define GDN_FLAG_LOG_GATE  2    /* alpha holds the log-space gate g; the kernels use alpha =
                                   expf(g) (CUDA's expf) */

/* Limits checked on the host. */
#define GDN_MAX_T 1024          /* draft tokens per request */

typedef struct gdn_problem {
    int32_t batch;               /* B >= 0 requests (B = 0: calls return GDN_OK, no launch) */
    int32_t heads;               /* H >= 1 */
    int32_t dk;                  /* key dim: 32, 64, 128 or 256 */
    int32_t dv;                  /* value dim: a multiple of 32, <= 128 or 256 */
    int32_t max_T;               /* uniform draft length (cu_seqlens NULL) or the ragged maximum, 0..GDN_MAX_T */
    int32_t qkv_dtype;           /* gdn_dtype of q, k, v */
    int32_t algo;                /* gdn_algo */
    int32_t flags;               /* GDN_FLAG_* bits; all other bits must be 0 */
    const int32_t *cu_seqlens;   /* device [batch+1] token-row offsets, or NULL (uniform) */
    const void *q;               /* device [N_tok][heads][dk], 16-byte aligned; may be NULL for
                                    the commit calls (gdn_commit, gdn_commit_layers,
                                    gdn_replay_commit), which read no q */
    const void *k;               /* device [N_tok][heads][dk], 16-byte aligned */
    const void *v;               /* device [N_tok][heads][dv], 16-byte aligned */
    const float *alpha;          /* device [N_tok][heads]: alpha, or g = log(alpha) with GDN_FLAG_LOG_GATE */
    const float *beta;           /* device [N_tok][heads] */
    float *pool;                 /* device [pool_slots][heads][dk][dv], 16-byte aligned */
    int64_t pool_slots;          /* >= batch */
    const int32_t *slot_ids;     /* device [batch], distinct, in [0, pool_slots) */
    int32_t *dev_err;            /* device int32 error word (GDN_DEVERR_* bits), or NULL */
    int64_t n_tok;               /* rows of q/k/v/alpha/beta/o.  Ignored for uniform input
                                    (batch*max_T); REQUIRED for ragged input: the kernels
                                    flag GDN_DEVERR_SEQLEN for a request whose rows
                                    [cu[r], cu[r+1]) do not lie in [0, n_tok) */
} gdn_problem;

/* o_t for every draft token of every unit.  o: device float32 (or, with
 * GDN_FLAG_O_BF16, bfloat16) [N_tok][heads][dv],
 * 16-byte aligned, must not overlap any input.  Reads the pool, never writes it. */
GDN_API gdn_status gdn_verify(const gdn_problem *p, void *o, cudaStream_t stream);

/* For every request r with accepted[r] > 0: pool[slot_ids[r]][h] <- state after
 * accepted[r] tokens, replayed from the checkpoint in that same slot (in place).
 * Requests with accepted[r] = 0 write nothing.  accepted: device int32 [batch]. */
GDN_API gdn_status gdn_commit(const gdn_problem *p, const int32_t *accepted, cudaStream_t stream);

/* gdn_verify and then gdn_commit with the same inputs, in one pass: each
 * checkpoint is read once, o is written for every token, the state once. */
GDN_API gdn_status gdn_verify_commit_fused(const gdn_problem *p, const int32_t *accepted,
                                           void *o, cudaStream_t stream);

/* Layer batches: the same calls for the n_layers problems of one step (one per
 * model layer), in as few launches as possible (the chunked kernel takes up to
 * 32 layers per launch, so the fill and drain of a launch are paid once for
 * all of them instead of once per layer).
 *
 * problems: host array of n_layers gdn_problem.  They must agree on the
 * request-level fields (batch, heads, dk, dv, max_T, qkv_dtype, algo,
 * cu_seqlens, slot_ids, pool_slots, and n_tok when ragged), else
 * GDN_ERR_LAYER_MISMATCH; each names its own q, k, v, alpha, beta, pool (that
 * layer's pool) and dev_err.  o: host array of n_layers device pointers, o[l]
 * for problem l as in gdn_verify.  accepted: one device array, shared by all
 * layers.  Each problem is validated as by the single-problem call; besides,
 * no layer's o, nor (commit, fused) its pool, may overlap another layer's
 * arrays (GDN_ERR_ALIAS).  The results equal those of the single-problem call
 * made once per layer.  n_layers = 0 launches nothing. */
GDN_API gdn_status gdn_verify_layers(const gdn_problem *problems, int32_t n_layers,
                                     void *const *o, cudaStream_t stream);
GDN_API gdn_status gdn_commit_layers(const gdn_problem *problems, int32_t n_layers,
                                     const int32_t *accepted, cudaStream_t stream);
GDN_API gdn_status gdn_verify_commit_fused_layers(const gdn_problem *problems, int32_t n_layers,
                                                  const int32_t *accepted, void *const *o,
                                                  cudaStream_t stream);

/* Greedy accepted lengths on the device, so that the commit needs no host round
 * trip: accepted[r] = the largest a in [0, T_r] such that
 *     draft_ids[c_r + t] == target_ids[c_r + t]   for every t < a,
 * with c_r, T_r the token rows of request r as for gdn_problem (cu_seqlens, or
 * r * max_T and max_T when cu_seqlens is NULL).  Speculative decoding keeps the
 * draft tokens that agree with the target model and rolls back to that prefix
 * (OCRia write-up, sections "Generate more tokens per target pass: speculative
 * decoding" and "Make speculative verification cheaper"); this is the greedy
 * form of that check.  The caller lines up both arrays so that row c_r + t
 * holds the draft id of the token fed at that row and the target's own choice
 * for it (a row that is always kept is passed with equal ids).
 *
 * draft_ids, target_ids: device int32 [n_tok] (uniform: batch * max_T rows);
 * accepted: device int32 [batch], written; it must not overlap the other
 * arrays.  A ragged request whose rows leave [0, n_tok) or whose length
 * leaves [0, max_T] sets GDN_DEVERR_SEQLEN in *dev_err and its accepted[r] is
 * not written.  batch = 0 launches nothing.  All pointers 4-byte aligned. */
GDN_API gdn_status gdn_accept_prefix(int32_t batch, int32_t max_T, const int32_t *cu_seqlens,
                                     int64_t n_tok, const int32_t *draft_ids,
                                     const int32_t *target_ids, int32_t *accepted,
                                     int32_t *dev_err, cudaStream_t stream);

/* ReplaySSM buffer (multi-step speculation).  ReplaySSM keeps a checkpoint of
 * the state next to a small buffer of recent inputs, computes outputs from
 * both, writes the full checkpoint only at periodic flushes, and rolls a
 * rejection back by moving the buffer pointer (OCRia write-up, section "Make
 * speculative verification cheaper").  Here pool[slot] is the checkpoint as
 * of the slot's last flush, and the slot's buffer holds the rows accepted
 * since then: rows slot * capacity + [0, len_in[slot]) of k, v, alpha, beta
 * (the layout of the token arrays, with pool_slots * capacity rows).
 *
 * A step, for request r in slot s with n = len_in[s]:
 *   1. the caller writes the step's draft rows of k, v, alpha, beta at buffer
 *      rows s * capacity + n + [0, T_r) (n + T_r <= capacity), and q as usual
 *      at rows cu[r] + [0, T_r) of p->q;
 *   2. gdn_replay_verify: o for the draft rows (rows cu[r] + t of o), from
 *      pool[s] and buffer rows [0, n + T_r); writes neither pool nor buffer;
 *   3. gdn_replay_commit with accepted[r] = a_r: keep = n + a_r.  If
 *      keep + max_T > capacity (a full next draft would not fit) the slot is
 *      flushed: pool[s][h] <- the state after buffer rows [0, keep) and
 *      len_out[s] = 0; otherwise the pool is not touched and len_out[s] = keep
 *      (rejected rows are overwritten by the next step's drafts);
 *   4. the caller swaps len_in and len_out for the next step.
 * Only the chunked kernel runs these calls (bf16 q/k/v, dk = dv = 128);
 * other shapes return GDN_ERR_UNSUPPORTED.  p->k, p->v, p->alpha and p->beta
 * are not used (the buffer holds those rows); every other field of p means
 * what it means for gdn_verify and gdn_commit.  A unit whose buffer does not
 * hold its rows (n < 0, n + T_r > capacity in verify, keep > capacity in
 * commit) sets GDN_DEVERR_REPLAY and is skipped; len_out[s] is then not
 * written.  len_out[s] is written for every named slot, by one thread;
 * entries of other slots are left as they are. */
typedef struct gdn_replay {
    int32_t capacity;            /* buffer rows per slot, >= max_T */
    int32_t reserved;            /* must be 0 */
    const void *k;               /* device [pool_slots * capacity][heads][dk], qkv_dtype, 16-byte aligned */
    const void *v;               /* device [pool_slots * capacity][heads][dv], 16-byte aligned */
    const float *alpha;          /* device [pool_slots * capacity][heads] */
    const float *beta;           /* device [pool_slots * capacity][heads] */
    const int32_t *len_in;       /* device [pool_slots]: rows buffered in each slot */
    int32_t *len_out;            /* device [pool_slots]: written by gdn_replay_commit; must not
                                    overlap len_in or any other array */
} gdn_replay;

GDN_API gdn_status gdn_replay_verify(const gdn_problem *p, const gdn_replay *rb, void *o,
                                     cudaStream_t stream);
GDN_API gdn_status gdn_replay_commit(const gdn_problem *p, const gdn_replay *rb,
                                     const int32_t *accepted, cudaStream_t stream);

/* Commit the previous step, then verify the next one, in one pass over each
 * checkpoint (OCRia write-up, section "Make speculative verification
 * cheaper": rollback keeps the accepted prefix; in an engine the accepted
 * lengths of a step are known only after all its layers have verified, so a
 * layer's commit of step n - 1 can run at its verify of step n).
 *
 * For every request r and head h, with S the state in pool[slot_ids[r]][h]:
 *   1. if prev->accepted[r] = a > 0: S <- the state after the first a rows of
 *      the previous step replayed from S, written back to the slot (as
 *      gdn_commit with that step's problem would);
 *   2. o <- the outputs of this step's drafts from S (as gdn_verify would).
 * The previous step's own W (a by-product of its call, written to its `w`) is
 * what makes step 1 a single rank-a update: no products of the checkpoint.
 *
 *   p     this step: everything gdn_verify takes.  bf16 q/k/v, dk = dv = 128,
 *         1 <= max_T <= 16 (GDN_ERR_UNSUPPORTED otherwise); AUTO or GDN_ALGO_CHUNK.
 *   prev  the previous step of the same requests (same batch, heads, slot ids),
 *         or NULL for the first step (nothing is committed).
 *   o     as gdn_verify.
 *   w     device float32 [N_tok][heads][dv], 16-byte aligned, written: this
 *         step's W, for the next call's prev->w (the caller alternates two
 *         buffers).  Must not overlap any other array of the call.
 * Device errors: prev->accepted[r] outside [0, T_prev,r] sets
 * GDN_DEVERR_ACCEPTED, bad previous row offsets GDN_DEVERR_SEQLEN; the unit is
 * skipped (no write, no outputs). */
typedef struct gdn_prev_step {
    const int32_t *cu_seqlens;   /* device [batch+1] row offsets of the previous step, or NULL (uniform max_T) */
    int32_t max_T;               /* its uniform length, or its ragged maximum; 0..16 */
    int32_t reserved;            /* must be 0 */
    int64_t n_tok;               /* rows of its arrays (ragged; ignored when cu_seqlens is NULL) */
    const void *k;               /* device, its k [n_tok][heads][dk], 16-byte aligned */
    const float *alpha;          /* device, its alpha (or g with GDN_FLAG_LOG_GATE) [n_tok][heads] */
    const float *w;              /* device, the w its call wrote [n_tok][heads][dv], 16-byte aligned */
    const int32_t *accepted;     /* device [batch]: its accepted lengths */
} gdn_prev_step;

GDN_API gdn_status gdn_commit_verify(const gdn_problem *p, const gdn_prev_step *prev, void *o,
                                     float *w, cudaStream_t stream);

/* Attention layers.  The other layers of a hybrid model keep keys and values
 * in a paged cache.  A step has the same requests and rows as the GDN calls
 * (uniform max_T, or cu_seqlens); kv_len[r] tokens of request r are in the
 * cache before it, and its row t (0 <= t < T_r) is the token at place
 * c = kv_len[r] + t.  Place c of request r lies in page
 * page_table[r][c / page_size], row c % page_size.  A rejected draft is rolled
 * back by leaving kv_len where it was: kv_len[r] += accepted[r] after a step,
 * and the next step overwrites the rejected rows.
 *
 * Layout: k_pages and v_pages are [n_pages][kv_heads][page_size][head_dim],
 * consecutive pages page_stride elements apart (>= kv_heads * page_size *
 * head_dim, so that both may lie in one allocation).  Query head h reads key
 * head h / (q_heads / kv_heads). */
#define GDN_ATTN_MAX_T 65536    /* rows per request of the two attention calls */

typedef struct gdn_attn {
    int32_t batch;               /* B >= 0 requests (B = 0: calls return GDN_OK, no launch) */
    int32_t q_heads;             /* a multiple of kv_heads, at most 65536; max_T * (q_heads / kv_heads) at most 2^30 */
    int32_t kv_heads;            /* >= 1 */
    int32_t head_dim;            /* 32, 64, 128 or 256 */
    int32_t max_T;               /* uniform rows per request (cu_seqlens NULL) or the ragged maximum, 0..GDN_ATTN_MAX_T;
                                    the kernel is chosen by it, so keep it as small as the rows allow */
    int32_t dtype;               /* gdn_dtype of q, k, v, the pages and o */
    int32_t page_size;           /* 16, 32, 64, 128 or 256 */
    int32_t max_pages;           /* columns of page_table; max_pages * page_size <= 2^31 - 1 */
    int32_t window;              /* 0: every place up to the row's own; W > 0: the last W of them, itself among them */
    int32_t sinks;               /* first places that stay visible under a window (0 without one) */
    float scale;                 /* factor on q.k, finite and above 0 (1 / sqrt(head_dim) in most models) */
    int32_t reserved;            /* must be 0 */
    const int32_t *cu_seqlens;   /* device [batch+1] token-row offsets, or NULL (uniform) */
    int64_t n_tok;               /* rows of q/k/v/o: REQUIRED for ragged input, ignored for uniform */
    void *k_pages;               /* device, 16-byte aligned; written by gdn_rope_append only */
    void *v_pages;               /* device, 16-byte aligned; written by gdn_rope_append only */
    int64_t n_pages;             /* 1 .. 2^31 - 1 */
    int64_t page_stride;         /* elements from a page to the next; a multiple of 16 bytes, at most 2^36,
                                    and n_pages * page_stride at most 2^56 */
    const int32_t *page_table;   /* device [batch][max_pages]; entries no row needs are not read */
    const int32_t *kv_len;       /* device [batch]: tokens in the cache before this step */
    int32_t *dev_err;            /* device int32 error word (GDN_DEVERR_* bits), or NULL */
} gdn_attn;

/* Rotary positions.  The first rot_dim elements of a head are rotated, the
 * rest pass unchanged.  Pair i of rot_dim / 2 is (x, y) = elements (i, i +
 * rot_dim / 2), or (2i, 2i + 1) when interleaved; with angle a = p *
 * inv_freq[i], p = positions[row] (or the row's place c when NULL),
 *     x' = mscale (x cos a - y sin a),   y' = mscale (x sin a + y cos a).
 * Scalings for long contexts are choices of inv_freq and mscale. */
typedef struct gdn_rope {
    int32_t rot_dim;             /* a multiple of 16, 16 .. head_dim */
    int32_t interleaved;         /* 0: halves, 1: neighbours */
    float mscale;                /* factor on cosine and sine, finite (1 without scaling) */
    int32_t reserved;            /* must be 0 */
    const float *inv_freq;       /* device float32 [rot_dim / 2]: radians per position */
    const int32_t *positions;    /* device int32 [N_tok], or NULL: the row's place in the cache */
} gdn_rope;

/* One step's rows: q_out <- rotated q, and the rotated k and the v of each row
 * to its place in the pages.
 *   q      device [N_tok][q_heads][head_dim], q_stride elements from a row to the next
 *   k, v   device [N_tok][kv_heads][head_dim], k_stride and v_stride elements apart
 *          (strides >= the row, multiples of 16 bytes, at most 2^36, and N_tok times a
 *          stride at most 2^56: slices of one projection's output)
 *   q_out  device [N_tok][q_heads][head_dim], contiguous; overlaps nothing else of the call
 * All 16-byte aligned.  A request with a bad kv_len or bad row offsets is skipped; a row
 * whose page id is outside [0, n_pages) gets its q_out and sets GDN_DEVERR_PAGE.  No two rows
 * of a call may share a place (a shared page that one of them writes is a precondition
 * violation). */
GDN_API gdn_status gdn_rope_append(const gdn_attn *p, const gdn_rope *rope, const void *q,
                                   int64_t q_stride, const void *k, int64_t k_stride,
                                   const void *v, int64_t v_stride, void *q_out,
                                   cudaStream_t stream);

/* Attention of the step's rows over the cache, which holds the step's own
 * keys and values already.  Row t of request r at place c = kv_len[r] + t sees
 * the places j <= c with (window = 0, or j > c - window, or j < sinks):
 *     o = sum_j e_j v_j / sum_j e_j,   e_j = exp(scale q.k_j - m),   m = max_j scale q.k_j
 *   q    device [N_tok][q_heads][head_dim], q_stride elements apart, 16-byte aligned
 *   o    device [N_tok][q_heads][head_dim], contiguous, dtype, 16-byte aligned
 *   lse  device float32 [N_tok][q_heads]: m + log(sum_j e_j), or NULL
 *   workspace  device, 16-byte aligned, at least gdn_paged_attn_workspace(p)
 *        bytes; one per stream.  Its first 16 KB have to be zero when it is
 *        first used, and again after a GDN_DEVERR_TIMEOUT: they hold counters,
 *        which every call leaves at zero (and what a call writes for itself,
 *        which no later call reads).
 * o, lse and the workspace overlap nothing else of the call.  Sums and the
 * softmax's statistics are 32-bit.  The weights e_j are rounded to bf16 for the
 * products with v where dtype is bf16, head_dim 64 or 128 and max_T * (q_heads /
 * kv_heads) above 16, and carried to 2^-16 elsewhere: a token's output as a single
 * row and within a draft may differ by a rounding of its weights.  Keys and values at places that no row of a
 * request sees are never used, whatever they hold.  An infinite value at a place
 * that a row sees makes that element of the row's output infinite; a NaN, or
 * infinities of both signs, make it NaN, and so may an infinite value whose
 * weight is below 2^-126.  A request with a bad kv_len or bad row offsets is
 * skipped (nothing is written for it); a page whose id is outside [0, n_pages)
 * sets GDN_DEVERR_PAGE and reads as zeros. */
GDN_API gdn_status gdn_paged_attn(const gdn_attn *p, const void *q, int64_t q_stride, void *o,
                                  float *lse, void *workspace, int64_t workspace_bytes,
                                  cudaStream_t stream);

/* Bytes of workspace that gdn_paged_attn needs for p (host only, no CUDA
 * call; depends on sizes and dtype, not on lengths), or -1 when p's sizes fail
 * validation. */
GDN_API int64_t gdn_paged_attn_workspace(const gdn_attn *p);

/* Linear attention with a decay for each head: layers that keep, like GDN
 * layers, a state per request and head, but only let it decay and add to it.  With S
 * the dk x dv state of one unit (request r, head h; the tile layout of the pool above) and
 * row t of the request,
 *
 *     S_t = e^{g_t} S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t
 *
 * g is the logarithm of the decay, at most 0 in most models (0: none, -infinity: the state
 * before is multiplied by 0): a constant of each head (decay_stride = 0), or given for each row.
 * Requests, rows and slots are those of the GDN calls, with up to GDN_ATTN_MAX_T rows a request:
 * single tokens, drafts and prompts.
 *
 * Products, sums and states are 32-bit, but for calls with bfloat16 rows, dk 64 or 128 and dv a
 * multiple of 64, which round states and weights for the tensor cores:
 *   gdn_linear_verify with max_T of 2 to 47: for o to two bfloat16 terms each, off by 2^-17 at most;
 *   all calls with max_T of 48 or more: for o to bfloat16 (2^-8), which o is itself, and what is added to
 *   a state to two bfloat16 terms;
 * so a row's o and a state may differ by such roundings from those of calls with other max_T.  Calls
 * with max_T of 48 or more of that kind let a value, key or query that is not finite make outputs of its
 * request and head not finite from the row's block of 128 rows on, the block's earlier rows among them;
 * all others from its own row on.
 *
 * Over blocks of up to 128 rows, the decay from one row (or the state before) to a later one is a float32, the
 * exponential of its logarithms' sum: where that leaves float32 it is 0 or infinite, even if what it
 * multiplies would bring it back.  Positive logarithms are allowed.  Calls of the second kind may take five
 * times as long where sums of theirs over up to 32 rows exceed 4 and leave -20 to 20. */
typedef struct gdn_linear {
    int32_t batch;               /* B >= 0 requests (B = 0: calls return GDN_OK, no launch) */
    int32_t heads;               /* H >= 1: states, and heads of v and o */
    int32_t k_heads;             /* heads of q and k, divides H: head h reads head h / (H / k_heads) */
    int32_t dk;                  /* 32, 64, 128 or 256 */
    int32_t dv;                  /* a multiple of 32, 32 .. 256 */
    int32_t max_T;               /* uniform rows per request (cu_seqlens NULL) or the ragged maximum, 0..GDN_ATTN_MAX_T;
                                    the kernel is chosen by it, so keep it as small as the rows allow */
    int32_t dtype;               /* gdn_dtype of q, k, v and o */
    float scale;                 /* factor on o, finite */
    const int32_t *cu_seqlens;   /* device [batch+1] token-row offsets, or NULL (uniform) */
    int64_t n_tok;               /* rows of the arrays: REQUIRED for ragged input, ignored for uniform */
    const void *q;               /* device [N_tok][k_heads][dk], q_stride elements from a row to the next; may be
                                    NULL for gdn_linear_commit */
    const void *k;               /* device [N_tok][k_heads][dk], k_stride elements apart */
    const void *v;               /* device [N_tok][heads][dv], v_stride elements apart */
    int64_t q_stride;            /* each at least the row, a multiple of 16 bytes, at most 2^36, and */
    int64_t k_stride;            /*   N_tok times a stride at most 2^56; pointers 16-byte aligned */
    int64_t v_stride;
    const float *log_decay;      /* device float32 [N_tok][heads], decay_stride elements apart, or [heads] */
    int64_t decay_stride;        /* 0: one row for all; else at least heads, at most 2^36 */
    float *pool;                 /* device float32 [pool_slots][heads][dk][dv], 16-byte aligned */
    int64_t pool_slots;          /* >= batch */
    const int32_t *slot_ids;     /* device [batch], distinct, in [0, pool_slots) */
    int32_t *dev_err;            /* device int32 error word (GDN_DEVERR_* bits), or NULL */
} gdn_linear;

/* o for every row from the states in the pool, which stays as it is (drafts).
 * o: device dtype [N_tok][heads][dv], contiguous, 16-byte aligned; it overlaps nothing else.
 * A request with a bad slot or bad row offsets is skipped, here and below. */
GDN_API gdn_status gdn_linear_verify(const gdn_linear *p, void *o, cudaStream_t stream);

/* pool[slot_ids[r]] <- the states after the first accepted[r] rows, for every request with
 * accepted[r] > 0 (device int32 [batch], in [0, T_r]); all other slots stay as they are. */
GDN_API gdn_status gdn_linear_commit(const gdn_linear *p, const int32_t *accepted,
                                     cudaStream_t stream);

/* Both in one pass, of all rows: o for every row, and the states after the last one (single
 * tokens, prompts).  A request without rows keeps its state. */
GDN_API gdn_status gdn_linear_step(const gdn_linear *p, void *o, cudaStream_t stream);

/* Accepted lengths and next tokens of sampled drafts, on the device (gdn_accept_prefix
 * is the greedy form).  Rows are those of the step that verified the drafts: row 0 of a
 * request is its last token, which is always kept, and row t >= 1 holds a draft, x = draft_ids[row].
 * Row t of target_probs is the target model's distribution after row t, so a draft at row t
 * is judged by row t - 1; row t - 1 of draft_probs is the distribution that it was drawn
 * from, q (NULL: drafts that were looked up, each with q = 1).  In the order of the rows,
 * draft x stays if
 *     u_accept[row] q(x) < p(x)
 * (compared without rounding), and the first that does not ends the request's rows:
 *     accepted[r] = 1 + the drafts that stay       (0 for a request without rows)
 * The next token follows the last row kept: drawn from max(p - q, 0) there if a
 * draft did not stay, from p if all did (and if p <= q everywhere).  With weights w_i in whole
 * units of 2^-44 (p and q rounded down to them first; NaN and what is below 0 counts as 0, above
 * 1 as 1), W their sum and U = floor(2^31 u_sample[r]), it is the lowest id i with
 *     w_0 + ... + w_i > floor(U W / 2^31).
 * All sums are of integers: the result is the same on every run, whatever the order.
 *
 * A draft id outside [0, vocab) does not stay, sets GDN_DEVERR_TOKEN, and the next token is
 * drawn as for any other; so does a row of p without any weight, whose next_ids is -1. */
#define GDN_MAX_VOCAB 262144

typedef struct gdn_sample {
    int32_t batch;               /* B >= 0 */
    int32_t max_T;               /* uniform rows per request (cu_seqlens NULL) or the ragged maximum, 0..GDN_MAX_T */
    int32_t vocab;               /* 1 .. GDN_MAX_VOCAB */
    int32_t reserved;            /* must be 0 */
    const int32_t *cu_seqlens;   /* device [batch+1] row offsets, or NULL (uniform) */
    int64_t n_tok;               /* rows: REQUIRED for ragged input, ignored for uniform */
    const int32_t *draft_ids;    /* device [N_tok]; a request's first is not read */
    const float *target_probs;   /* device [N_tok][vocab], target_stride elements from a row to the next */
    int64_t target_stride;       /* >= vocab, at most 2^36 */
    const float *draft_probs;    /* device [N_tok][vocab], draft_stride elements apart, or NULL */
    int64_t draft_stride;
    const float *u_accept;       /* device [N_tok], in [0, 1); a request's first is not read */
    const float *u_sample;       /* device [batch], in [0, 1); other values are taken to 0 and to 1 - 2^-31 */
    int32_t *dev_err;            /* device int32 error word, or NULL */
} gdn_sample;

/* accepted, next_ids: device int32 [batch], written; they overlap nothing else.  accepted is what the
 * commit calls take, next_ids the tokens to feed next (-1 for a request without rows).  A
 * request whose rows leave [0, n_tok) or [0, max_T] sets GDN_DEVERR_SEQLEN and gets neither. */
GDN_API gdn_status gdn_accept_sample(const gdn_sample *p, int32_t *accepted, int32_t *next_ids,
                                     cudaStream_t stream);

/* The next step of the requests of a paged cache, from lengths that only the device knows (the
 * rows that were accepted): the lengths move, pages that are no longer needed go back to a
 * free list and new ones come from it, and the row offsets, slots and positions that the
 * step's calls read are written.  For request r in order, with a = accepted[r]:
 *   length   l = kv_len[r] + a, or 0 if done[r] (it has ended, all its pages go back)
 *   rows     T = rows[r], or max_T when rows is NULL; 0 if done[r]
 *   pages    n = ceil((l + T) / page_size).  Of its held[r] pages, those in columns n and
 *            on of its row of the page table go back, behind the free list's last (in the
 *            order of requests and columns).  If n > held[r], n - held[r] pages come from the
 *            list's end, the last one first, into columns held[r] and on, after all pages
 *            of the call have gone back.
 * A request gets its pages if the list has enough for all that are wanted up to and with its
 * own (one that wants none goes on in any case).  One that does not keeps the pages it holds,
 * has no rows in this step and sets GDN_DEVERR_NO_PAGES; its length moves all the same, so plan
 * again, with accepted NULL, when there are pages.
 *   kv_len_out[r] = l      held_out[r] = n (or held[r])    free_count_out = pages left
 *   cu_seqlens = the rows' offsets (what the GDN, linear and attention calls take, with
 *            n_tok = an upper bound)
 *   slots[row] = page * page_size + row in the page, and positions[row] = l + t, for every row
 *            of the step; what lies behind the last row is left as it was
 * Device errors, each with no rows for the request: rows outside [0, max_T]
 * (GDN_DEVERR_SEQLEN), kv_len < 0 or held outside [0, max_pages] (GDN_DEVERR_KV_LEN), a < 0 or more
 * places used than the held pages have (GDN_DEVERR_ACCEPTED): its length and pages
 * stay (of one that has ended only held is looked at); l + T above max_pages * page_size (GDN_DEVERR_KV_LEN): its length moves, T counts
 * as 0.  A free count outside [0, n_pages], or more pages going back than the list has room for, sets
 * GDN_DEVERR_PAGE, and no length or page moves and no request has rows. */
typedef struct gdn_pages {
    int32_t batch;               /* B >= 0 (0: GDN_OK, no launch, nothing written) */
    int32_t max_T;               /* 0..GDN_ATTN_MAX_T; batch * max_T at most 2^31 - 1 */
    int32_t page_size;           /* 16, 32, 64, 128 or 256 */
    int32_t max_pages;           /* columns of page_table, >= 1; max_pages * page_size <= 2^31 - 1, batch * max_pages too */
    int64_t n_pages;             /* entries of free_pages, 1 .. 2^31 - 1 */
    const int32_t *rows;         /* device [batch], or NULL */
    const int32_t *accepted;     /* device [batch], or NULL (0 each) */
    const int32_t *done;         /* device [batch], not 0: ended; or NULL */
    const int32_t *kv_len;       /* device [batch] */
    const int32_t *held;         /* device [batch]: pages of each request */
    const int32_t *free_count;   /* device [1] */
    int32_t *kv_len_out;         /* device [batch]; each of the three may be its input's array, */
    int32_t *held_out;           /* device [batch];   or one that overlaps nothing else */
    int32_t *free_count_out;     /* device [1] */
    int32_t *free_pages;         /* device [n_pages]: the free list, its first free_count entries */
    int32_t *page_table;         /* device [batch][max_pages] */
    int32_t *cu_seqlens;         /* device [batch+1], written */
    int64_t *slots;              /* device [max_rows], 8-byte aligned, written; or NULL */
    int32_t *positions;          /* device [max_rows], written; or NULL */
    int64_t max_rows;            /* entries of slots and positions, >= 0: rows from there on are not
                                    written and set GDN_DEVERR_SEQLEN */
    int32_t *dev_err;            /* device int32 error word, or NULL */
} gdn_pages;

GDN_API gdn_status gdn_plan_pages(const gdn_pages *p, cudaStream_t stream);

/* Waits for `stream`, copies *p->dev_err to *host_code (0 when dev_err is NULL).
 * Returns GDN_ERR_DEVICE_ARG when the word is non-zero, GDN_OK when it is zero. */
GDN_API gdn_status gdn_read_device_error(const gdn_problem *p, cudaStream_t stream,
                                         int32_t *host_code);

/* The same for the attention calls: of *p only dev_err is read. */
GDN_API gdn_status gdn_read_attn_error(const gdn_attn *p, cudaStream_t stream, int32_t *host_code);

/* The same for any error word (device int32, or NULL: no error). */
GDN_API gdn_status gdn_read_error(const int32_t *dev_err, cudaStream_t stream, int32_t *host_code);

/* Self-check of the bounded waits (diagnostic; not part of a decode step).
 * The chunked kernel waits on shared-memory barriers for its copies and
 * products, and gives up after about two seconds with GDN_DEVERR_TIMEOUT
 * rather than hang.  This call runs that same wait in one block, on a barrier
 * that nothing completes: after about two seconds the block ORs
 * GDN_DEVERR_TIMEOUT into *dev_err and exits, and the CUDA context stays
 * usable.  Asynchronous on `stream` (one SM is busy meanwhile).
 * dev_err: device int32, caller-owned, 4-byte aligned, not NULL (else
 * GDN_ERR_NULL_PTR / GDN_ERR_ALIGN before any CUDA call). */
GDN_API gdn_status gdn_selftest_wait_timeout(int32_t *dev_err, cudaStream_t stream);

/* The algo that AUTO resolves to for this problem (host only, no CUDA call),
 * or -1 when the shape fails validation. */
GDN_API int32_t gdn_select_algo(const gdn_problem *p);

/* Static, never NULL. */
GDN_API const char *gdn_status_string(gdn_status s);

/* Text of the last CUDA error seen by this thread ("" if none). */
GDN_API const char *gdn_last_error_string(void);

/* Library version, e.g. "0.1.0". */
GDN_API const char *gdn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
