// Shared device-side pieces of the attention calls over a paged key/value
// cache: the kernel argument block, the division of a call's work among the
// blocks, and the places of partial results.
//
// Work.  A unit is (request r, query tile qt, key head h): ROWS query rows,
// row i of the tile being (token t, head g of the group) with qt * ROWS + i =
// t * G + g, so that every key and value read serves all G query heads that
// share it.  A unit's key tiles (KT places each) cover the places that some row
// of it sees, without a gap: under a window the first `sinks` places (rounded up
// to ALIGN of them), then those from the first row's window (rounded down) to the last
// row's own place.  All
// units' tiles in order (request, query tile, key head, tile) form one line of
// N tiles, and worker c of P takes tiles [c N / P, (c + 1) N / P): equal work
// whatever the requests' lengths, which only the device knows.  A unit's start and
// end take time too, so each has EXTRA places on the line before its tiles, in
// which nothing is done.  A unit that
// lies in one worker's range is finished there; one that spans several leaves
// a partial (unnormalised sums, running maximum, total) per worker.  They are joined
// by the block that writes the last of them (on the tensor cores in groups, level by
// level) or by combine_kernel, as launch_attn chooses; in the order of the workers
// either way, so results do not depend on timing.  A worker has at most two partials:
// the end of a unit begun earlier (slot 2c) and the beginning of one finished later
// (slot 2c + 1).
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn.h"

namespace gdn {

struct AttnArgs {
    int B, Hq, Hkv, G, hd, max_T;
    uint32_t g_magic, g_shift;  // n / G = umulhi(n, g_magic) >> g_shift for n < 2^31, G > 1
    int page_shift;          // log2 of the page size
    int max_pages;
    int window, sinks;       // window = 0: none
    float scale_log2;        // scale * log2(e): the softmax runs in powers of two
    long long n_tok;
    const int32_t *cu_seqlens;
    const void *k, *v;
    long long n_pages, page_stride;  // page_stride in elements
    const int32_t *page_table;
    const int32_t *kv_len;
    int32_t *dev_err;
    const void *q;
    long long q_stride;
    void *o;
    float *lse;
    float *part;             // 2P partial slots of ROWS * (hd + 2) floats
    int4 *desc;              // [P][2]: which unit worker c leaves unfinished
    int *count;              // [kAttnLevels][P], zero between calls: partials written of the unit
                             // that begins in worker c (on tensor cores, of the group that
                             // does, by level); NULL: combine_kernel joins them, by desc
};

__device__ __forceinline__ int div_group(const AttnArgs &a, int n) {
    return a.G == 1 ? n : (int)(__umulhi((unsigned)n, a.g_magic) >> a.g_shift);
}

// One request's rows and place in the cache; ok = false: skipped.
struct AttnReq {
    int row0, T, ctx;
    bool ok;
};

__device__ __forceinline__ AttnReq load_request(const AttnArgs &a, int r, bool report) {
    AttnReq q;
    long long c1;
    if (a.cu_seqlens) {
        q.row0 = a.cu_seqlens[r];
        c1 = a.cu_seqlens[r + 1];
    } else {
        q.row0 = r * a.max_T;
        c1 = (long long)q.row0 + a.max_T;
    }
    q.ctx = a.kv_len[r];
    const long long T = c1 - q.row0;
    int err = 0;
    if (T < 0 || T > a.max_T || q.row0 < 0 || c1 > a.n_tok) err |= GDN_DEVERR_SEQLEN;
    q.T = (int)T;
    if (q.ctx < 0 || (!err && (long long)q.ctx + T > ((long long)a.max_pages << a.page_shift)))
        err |= GDN_DEVERR_KV_LEN;
    if (err && report && a.dev_err) atomicOr(a.dev_err, err);
    q.ok = err == 0;
    return q;
}

// The places that query tile qt of a request sees, numbered without a gap: number v is
// place v below `first`, place v + shift from there on (no window, or one that reaches
// the sinks: shift = 0).  The rows' own places and the sinks are in these numbers too.
struct TileSpan {
    int n;             // tiles of KT numbers, 0 when the query tile has no rows
    int first, shift;
    int pmin, pmax;    // of the first and the last row
    int sinks;
};

// align: a power of two that divides KT and the page size (or is divided by it).
template <int ROWS, int KT>
__device__ __forceinline__ TileSpan tile_span(const AttnArgs &a, int T, int ctx, int qt, int align) {
    TileSpan s;
    const int first = qt * ROWS, rows = T * a.G;  // below 2^31: checked on the host
    if (first >= rows) {
        s.n = s.first = s.shift = s.pmin = s.pmax = s.sinks = 0;
        return s;
    }
    const int last = min(ROWS, rows - first) + first - 1;
    const int pmin = ctx + div_group(a, first), pmax = ctx + div_group(a, last);
    s.first = s.shift = 0;
    if (a.window) {
        const int lo = max(pmin - a.window + 1, 0) & -align;
        const int keep = (min(a.sinks, lo) + align - 1) & -align;
        if (keep < lo) {
            s.first = keep;
            s.shift = lo - keep;
        }
    }
    s.pmin = pmin - s.shift;
    s.pmax = pmax - s.shift;
    s.sinks = a.sinks;
    s.n = s.pmax / KT + 1;
    return s;
}

__device__ __forceinline__ int place_of(const TileSpan &s, int v) {
    return v + (v >= s.first ? s.shift : 0);
}

// Whether the row whose own place is number p sees number v.
__device__ __forceinline__ bool row_sees(const AttnArgs &a, const TileSpan &s, int p, int v) {
    return v <= p && (a.window == 0 || v > p - a.window || v < s.sinks);
}

// Whether some row sees some number of [v0, v1], or every row all of them.
__device__ __forceinline__ bool some_see(const AttnArgs &a, const TileSpan &s, int v0, int v1) {
    return v0 <= s.pmax && (a.window == 0 || v1 > s.pmin - a.window || v0 < s.sinks);
}
__device__ __forceinline__ bool all_see(const AttnArgs &a, const TileSpan &s, int v0, int v1) {
    return v1 <= s.pmin && (a.window == 0 || v0 > s.pmax - a.window || v1 < s.sinks);
}

// A worker's current run of tiles [i0, i1) of one unit.
struct Segment {
    int r, qt, h;
    AttnReq req;
    TileSpan span;
    int i0, i1;
};

// Shared-memory scratch of make_plan.
struct PlanScratch {
    long long warp_sum[32];
    long long x0, x1, total;
    long long off;   // of x0 within its entry
    int entry;       // (r, qt) that holds x0, as r * nq_max + qt
    int workers;
};

// A worker's position on the line of tiles.
struct Cursor {
    long long x, x1;   // next place of the line, end of the range
    long long off;     // of x within the entry
    int r, qt;
    int P;             // workers, and
    long long N;       // places of the line
};

// The range of worker c.
__device__ __forceinline__ void worker_range(int c, int P, long long N, long long &x0, long long &x1) {
    if (c >= P) {
        x0 = x1 = 0;
    } else if (N < (1 << 22)) {  // 32-bit products and quotients: c + 1 is below 2^10
        x0 = (unsigned)c * (unsigned)N / (unsigned)P;
        x1 = (unsigned)(c + 1) * (unsigned)N / (unsigned)P;
    } else {
        x0 = c * N / P;
        x1 = (c + 1) * N / P;
    }
}

// Every thread of the block calls it.  At least MIN_TILES places of the line to a worker:
// fewer, longer runs when there is little work.  Up to 32 entries (request, query tile) every
// warp adds them up for itself, an entry a lane, without a barrier; more are spread over
// the block.
template <int NT, int ROWS, int KT, int EXTRA, int MIN_TILES>
__device__ __forceinline__ Cursor make_plan(const AttnArgs &a, int c, int P, int align,
                                            PlanScratch *s, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nqm = a.max_T ? (a.max_T * a.G + ROWS - 1) / ROWS : 1;
    const unsigned E = (unsigned)a.B * nqm;  // below 2^31: checked on the host
    Cursor cur;
    if (E <= 32) {
        const int r = lane / nqm, qt = lane - r * nqm;
        long long sum = 0;
        if (lane < (int)E) {
            const AttnReq q = load_request(a, r, report && warp == 0 && qt == 0);
            const int n = q.ok ? tile_span<ROWS, KT>(a, q.T, q.ctx, qt, align).n : 0;
            sum = n ? (long long)(n + EXTRA) * a.Hkv : 0;
        }
        long long incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        cur.N = __shfl_sync(0xffffffffu, incl, 31);
        const long long by_size = (cur.N + MIN_TILES - 1) / MIN_TILES;
        cur.P = by_size < P ? (int)by_size : P;
        worker_range(c, cur.P, cur.N, cur.x, cur.x1);
        const unsigned here = __ballot_sync(0xffffffffu, cur.x >= incl - sum && cur.x < incl);
        const int src = here ? __ffs(here) - 1 : 0;
        cur.off = cur.x - __shfl_sync(0xffffffffu, incl - sum, src);
        cur.r = src / nqm;
        cur.qt = src - cur.r * nqm;
        return cur;
    }

    const unsigned chunk = (E + NT - 1) / NT;
    const unsigned e0 = min(tid * chunk, E), e1 = min(e0 + chunk, E);
    if (tid == 0) s->entry = -1;
    // Tiles of this thread's entries.
    long long sum = 0;
    for (unsigned e = e0; e < e1;) {
        const int r = (int)(e / nqm);
        int qt = (int)(e - r * nqm);
        const unsigned rend = (unsigned)(r + 1) * nqm;
        const AttnReq q = load_request(a, r, report && qt == 0);
        if (q.ok) {
            for (unsigned f = e; f < e1 && f < rend; ++f, ++qt) {
                const int n = tile_span<ROWS, KT>(a, q.T, q.ctx, qt, align).n;
                if (n == 0) break;
                sum += (long long)(n + EXTRA) * a.Hkv;
            }
        }
        e = rend;
    }
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) s->warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const long long w = lane < NT / 32 ? s->warp_sum[lane] : 0;
        long long wi = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, wi, d);
            if (lane >= d) wi += y;
        }
        s->warp_sum[lane] = wi - w;
        if (lane == 31) {
            const long long by_size = (wi + MIN_TILES - 1) / MIN_TILES;
            s->total = wi;
            s->workers = by_size < P ? (int)by_size : P;
            worker_range(c, s->workers, wi, s->x0, s->x1);
        }
    }
    __syncthreads();
    const long long x0 = s->x0, x1 = s->x1;
    const long long before = s->warp_sum[warp] + incl - sum;
    if (x1 > x0 && x0 >= before && x0 < before + sum) {  // exactly one thread
        long long at = before;
        for (unsigned e = e0; e < e1;) {
            const int r = (int)(e / nqm);
            int qt = (int)(e - r * nqm);
            const unsigned rend = (unsigned)(r + 1) * nqm;
            const AttnReq q = load_request(a, r, false);
            if (q.ok) {
                for (unsigned f = e; f < e1 && f < rend; ++f, ++qt) {
                    const int n = tile_span<ROWS, KT>(a, q.T, q.ctx, qt, align).n;
                    if (n == 0) break;
                    const long long m = (long long)(n + EXTRA) * a.Hkv;
                    if (x0 < at + m) {
                        s->entry = (int)f;
                        s->off = x0 - at;
                        e = e1;
                        break;
                    }
                    at += m;
                }
            }
            e = e < rend ? rend : e;
        }
    }
    __syncthreads();
    cur.N = s->total;
    cur.P = s->workers;
    cur.x = x0;
    cur.x1 = s->entry >= 0 ? x1 : x0;
    cur.off = s->entry >= 0 ? s->off : 0;
    cur.r = s->entry >= 0 ? s->entry / nqm : 0;
    cur.qt = s->entry >= 0 ? s->entry % nqm : 0;
    return cur;
}

// The next run of tiles of this worker; false, with g as it was, when its range is done.
template <int ROWS, int KT, int EXTRA>
__device__ __forceinline__ bool next_segment(const AttnArgs &a, int align, Cursor &cur,
                                             Segment &out) {
    while (cur.x < cur.x1) {
        Segment g;
        for (; cur.r < a.B; ++cur.r, cur.qt = 0) {
            g.req = load_request(a, cur.r, false);
            if (!g.req.ok) continue;
            g.span = tile_span<ROWS, KT>(a, g.req.T, g.req.ctx, cur.qt, align);
            if (g.span.n) break;  // a query tile with rows; else the next request's first
        }
        if (cur.r >= a.B) return false;
        const int n = g.span.n, m = n + EXTRA;
        g.r = cur.r;
        g.qt = cur.qt;
        g.h = (int)((unsigned long long)cur.off < (1ull << 32) ? (unsigned)cur.off / (unsigned)m
                                                               : cur.off / m);
        const int p0 = (int)(cur.off - (long long)g.h * m);
        const long long left = cur.x1 - cur.x;
        const int len = left < m - p0 ? (int)left : m - p0;
        g.i0 = max(p0 - EXTRA, 0);
        g.i1 = max(p0 + len - EXTRA, 0);
        cur.x += len;
        cur.off += len;
        if (cur.off >= (long long)m * a.Hkv) {
            cur.off = 0;
            ++cur.qt;
        }
        if (g.i1 > g.i0) {
            out = g;
            return true;
        }
    }
    return false;
}

// The worker that holds tile g of the line of N tiles.
__device__ __forceinline__ int worker_of(long long g, long long N, int P) {
    return (int)(((g + 1) * P - 1) / N);
}

// Slot of a segment that does not cover its unit.
__device__ __forceinline__ int part_slot(int c, const Segment &g) {
    return 2 * c + (g.i0 == 0 ? 1 : 0);
}

// Within a slot of ROWS rows: element (row, col) of the output, four columns together
// and then the next row, so that a thread a row (or a fragment) writes whole lines;
// then the maxima and the totals.
template <int ROWS>
__device__ __forceinline__ int part_at(int row, int col) {
    return ((col >> 2) * ROWS + row) * 4 + (col & 3);
}

// desc[c]: the unit whose beginning worker c holds and does not finish.  x is
// the line position after segment g (its last segment); one thread calls it.
__device__ __forceinline__ void write_desc(const AttnArgs &a, int c, const Segment &g, bool any,
                                           long long x, long long N, int P) {
    int4 d0 = make_int4(-1, 0, 0, 0), d1 = make_int4(0, 0, 0, 0);
    if (any && g.i0 == 0 && g.i1 < g.span.n) {
        d0 = make_int4(worker_of(x - g.i1 + g.span.n - 1, N, P), g.qt, g.h, g.req.row0);
        d1 = make_int4(g.req.T, 0, 0, 0);
    }
    a.desc[2 * c] = d0;
    a.desc[2 * c + 1] = d1;
}

__device__ __forceinline__ void put(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float4 x) {  // rounded once, to nearest even
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
}

// A running softmax state (maximum, total, outputs) and the addition of another.
template <int PER>
struct Partial {
    float m = -INFINITY, l = 0.f;
    float4 o[PER] = {};
    // o += f x, with m, l, o taken to the larger of the two maxima first.
    __device__ __forceinline__ void add(float xm, float xl, const float4 *x) {
        const float top = fmaxf(m, xm), base = top == -INFINITY ? 0.f : top;
        const float f = exp2f(m - base), g = exp2f(xm - base);
        m = top;
        l = l * f + xl * g;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            o[e].x = o[e].x * f + x[e].x * g;
            o[e].y = o[e].y * f + x[e].y * g;
            o[e].z = o[e].z * f + x[e].z * g;
            o[e].w = o[e].w * f + x[e].w * g;
        }
    }
};

// Partials w0, w0 + step, ... up to `last` of row `row`, PER column groups (of four) from cg on,
// CSTEP apart; the first is worker c's slot 2c + 1.  Four are in flight at a time.
template <int ROWS, int HD, int PER, int CSTEP>
__device__ __forceinline__ void add_partials(const AttnArgs &a, Partial<PER> &s, int c, int w0, int step,
                                             int last, int row, int cg) {
    constexpr int U = PER <= 4 ? 4 : 1;
    for (int w = w0; w <= last; w += U * step) {
        float m[U], l[U];
        float4 x[U][PER];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int wu = w + u * step;
            m[u] = -INFINITY;
            l[u] = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) x[u][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (wu > last) continue;
            const float *p = a.part + (long long)(wu == c ? 2 * c + 1 : 2 * wu) * ROWS * (HD + 2);
            m[u] = __ldcg(p + ROWS * HD + row);
            l[u] = __ldcg(p + ROWS * HD + ROWS + row);
#pragma unroll
            for (int e = 0; e < PER; ++e)
                x[u][e] = __ldcg(reinterpret_cast<const float4 *>(
                    p + part_at<ROWS>(row, 4 * (cg + e * CSTEP))));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) s.add(m[u], l[u], x[u]);
    }
}

// Called by all NT threads of a block that has written its partial of segment g (x: the
// line position after it): the block whose partial is the unit's last joins them.
template <typename T, int ROWS, int HD, int NT>
__device__ __forceinline__ void join_if_last(const AttnArgs &a, int c, const Segment &g, long long x,
                                             long long N, int P, int2 *shared) {
    __threadfence();
    __syncthreads();
    const int tid = threadIdx.x;
    if (tid == 0) {
        const long long begin = x - g.i1;  // of the unit's tiles
        const int first = worker_of(begin, N, P), last = worker_of(begin + g.span.n - 1, N, P);
        const bool all = atomicAdd(a.count + first, 1) == last - first;
        if (all) a.count[first] = 0;  // for the next call
        *shared = make_int2(all ? first : -1, last);
    }
    __syncthreads();
    const int first = shared->x, last = shared->y;
    if (first < 0) return;
    __threadfence();
    constexpr int PER = ROWS * HD / 4 > NT ? ROWS * HD / 4 / NT : 1, CSTEP = NT / ROWS;
    const int row = tid % ROWS, cg = tid / ROWS;
    if (cg >= HD / 4) return;  // more threads than vectors
    Partial<PER> s;
    add_partials<ROWS, HD, PER, CSTEP>(a, s, first, first, 1, last, row, cg);
    const int i = g.qt * ROWS + row;
    if (i >= g.req.T * a.G) return;
    const int t = div_group(a, i);
    const long long at = (long long)(g.req.row0 + t) * a.Hq + g.h * a.G + (i - t * a.G);
    const float inv = 1.f / s.l;
#pragma unroll
    for (int e = 0; e < PER; ++e)
        put(static_cast<T *>(a.o) + at * HD + 4 * (cg + e * CSTEP),
            make_float4(s.o[e].x * inv, s.o[e].y * inv, s.o[e].z * inv, s.o[e].w * inv));
    if (a.lse && cg == 0) a.lse[at] = (s.m + log2f(s.l)) * 0.69314718055994531f;
}

}  // namespace gdn
