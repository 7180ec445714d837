// Attention over a paged cache on the tensor cores (tcgen05): drafts of many
// query rows a key head, and prompt chunks (bf16, heads of 64 and 128).
//
// One block an SM, on tiles of 128 places.  A lane-parallel TMA
// warp streams keys and values, page by page, into a ring in shared memory
// (128-byte swizzle; a page that no row needs, or that does not exist, is asked
// for past the tensor's end and reads as zeros without traffic).  One thread
// issues the products: S = Q K^T with both operands in shared memory, O += P V with
// the weights P in tensor memory.  Two warpgroups do the softmax, a thread a row,
// each with its own S and O in tensor memory, so that the tensor cores work for
// one while the other is between its products:
//
//   WIDE (prompt chunks): a unit is 256 rows, 128 a warpgroup; both use each key
//     tile.  Bound by the tensor cores: 2 * 128^2 * HD * 2 flops a tile and
//     warpgroup.
//   otherwise (drafts, up to 128 rows a key head): both warpgroups have the same
//     128 rows and take the key tiles in turn, and their results are joined at the
//     end of a segment.  Bound by the cache's bytes; rows that are not there cost
//     tensor time that the stream leaves over.
//
// A row's maximum is replaced, and its output rescaled in tensor memory, only
// when it has grown by more than 2^8 (kLazy): the weights then stay below 2^8,
// which their float32 sums hold as exactly.  The weights are rounded to bf16 for
// the second product (its operands have one type); their total is summed
// before the rounding.
//
// Places that no row sees, and values that are not finite where some rows must
// not see them, would still reach the output as 0 * NaN.  In the tiles where
// any row's mask hides something (the ends of a unit) the warpgroups therefore
// clear them from the value tile first; the rows that do see such a value get it
// added at the end (add_unbounded).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "gdn_attn.cuh"
#include "gdn_launch.h"
#include "gdn_wait.cuh"

namespace gdn {
namespace {

constexpr int kKT = 128;       // places of a tile
constexpr int kThreads = 320;  // two softmax warpgroups, the TMA warp, the MMA warp
constexpr float kLazy = 8.f;
constexpr uint32_t kP = 64;    // TMEM column of P_w within S_w: two weights a column

template <int HD>
struct Cfg {
    static constexpr int kTile = kKT * HD * 2;     // bytes of a key (value, query) tile
    static constexpr int kBox = kKT * 128;         // bytes of 64 of its columns
    static constexpr int NS = HD == 128 ? 5 : 12;  // ring slots
    static constexpr int kTiles = (2 + NS) * kTile;  // queries, ring
    static constexpr uint32_t kO = 256;            // TMEM column of O_0 (S_0 at 0, S_1 at 128)
};

struct Bars {
    unsigned long long full[12], empty[12];
    unsigned long long s_full[2], p_ready[2], o_full[2], q_ready[2], clean[2], joined, drain;
};

struct Shared {
    Bars b;
    PlanScratch plan;
    uint32_t tmem;
    int dead;          // a wait gave up: every role leaves
    int poison[4];     // segment (mod 4) whose hidden places hold values that are not finite
    float m[2][kKT], l[2][kKT];
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint32_t bar(const unsigned long long &b) { return smem_addr(&b); }

__device__ __forceinline__ void arrive(uint32_t b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(b) : "memory");
}
__device__ __forceinline__ void arrive_expect(uint32_t b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(b), "r"(bytes)
                 : "memory");
}

// Bounded wait of one thread; false once any role of the block has given up.
__device__ __forceinline__ bool wait_one(uint32_t b, uint32_t parity, int *dead) {
    if (mbar_try_wait(b, parity)) return true;
    unsigned long long t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(b, parity)) return true;
        if ((it & 63) == 0) {
            if (*(volatile int *)dead) return false;
            const unsigned long long now = globaltimer();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitNs) *(volatile int *)dead = 1;
        }
    }
}
// The same by all 32 threads of a warp, with one answer.
__device__ __forceinline__ bool wait(uint32_t b, uint32_t parity, int *dead) {
    return __all_sync(0xffffffffu, wait_one(b, parity, dead));
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                       int c3, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(b)
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: rows of 128 bytes in groups of
// eight (sbo apart), column boxes lbo apart.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, bf16 operands, float32 accumulator, M = 128; A K-major, B K- or MN-major.
__host__ __device__ constexpr uint32_t idesc(uint32_t n, bool b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((n >> 3) << 17) |
           ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(b)
                 : "memory");
}
__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

#define GDN_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define GDN_W4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];\n"
        : GDN_R4(r, 0), GDN_R4(r, 4), GDN_R4(r, 8), GDN_R4(r, 12), GDN_R4(r, 16), GDN_R4(r, 20),
          GDN_R4(r, 24), GDN_R4(r, 28)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31, %32};\n" ::"r"(addr),
        GDN_W4(r, 0), GDN_W4(r, 4), GDN_W4(r, 8), GDN_W4(r, 12), GDN_W4(r, 16), GDN_W4(r, 20),
        GDN_W4(r, 24), GDN_W4(r, 28)
        : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Every row of the unit sees all places [j0, j0 + 128).
__device__ __forceinline__ bool tile_full(const AttnArgs &a, const TileSpan &s, int j0) {
    return j0 + kKT - 1 <= s.pmin &&
           (a.window == 0 || j0 > s.pmax - a.window || j0 + kKT - 1 < a.sinks);
}

struct Launch {
    AttnArgs a;
    CUtensorMap k, v;
};

// ---------------------------------------------------------------- the TMA warp

template <int HD, bool WIDE>
__device__ __forceinline__ void load_role(const Launch &L, Shared &s, uint32_t ring, Cursor cur,
                                          int lane, uint32_t &issued) {
    using C = Cfg<HD>;
    constexpr int ROWS = WIDE ? 256 : 128;
    const AttnArgs &a = L.a;
    const int rows_box = min(1 << a.page_shift, kKT);  // places of a TMA box
    const int boxes = kKT / rows_box;
    uint32_t pos = 0;
    Segment g;
    // This lane's page of tile i: its row and number, or n_pages (nothing needed, or no page).
    auto page_of = [&](int i, int &row) -> int {
        const int j = tile_place<kKT>(g.span, i) + lane * rows_box;
        row = j & ((1 << a.page_shift) - 1);
        const TileSpan &sp = g.span;
        if (lane >= boxes || i >= g.i1 || j > sp.pmax ||
            !(a.window == 0 || j + rows_box - 1 > sp.pmin - a.window || j < a.sinks))
            return (int)a.n_pages;
        const int page = a.page_table[(long long)g.r * a.max_pages + (j >> a.page_shift)];
        if (page >= 0 && page < a.n_pages) return page;
        if (a.dev_err) atomicOr(a.dev_err, GDN_DEVERR_PAGE);
        return (int)a.n_pages;
    };
    auto issue = [&](const CUtensorMap *map, int page, int row) -> bool {
        const uint32_t slot = pos % C::NS, round = pos / C::NS;
        ++pos;
        if (!wait(bar(s.b.empty[slot]), (round & 1) ^ 1, &s.dead)) return false;
        const uint32_t f = bar(s.b.full[slot]);
        if (lane == 0) arrive_expect(f, C::kTile);
        __syncwarp();
        if (lane < boxes) {
            const uint32_t dst = ring + slot * C::kTile + lane * rows_box * 128;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h)
                tma_4d(dst + h * C::kBox, map, 64 * h, row, g.h, page, f);
        }
        issued = pos;
        return true;
    };
    while (next_segment<ROWS, kKT>(a, cur, g)) {
        int row_n, next = page_of(g.i0, row_n);
        int p0 = 0, r0 = 0, p1 = 0, r1 = 0, held = 0;  // pages of tiles whose values are to come
        int ik = g.i0;
        auto keys = [&]() -> bool {
            const int page = next, row = row_n;
            next = page_of(++ik, row_n);
            if (held++ == 0) {
                p0 = page;
                r0 = row;
            } else {
                p1 = page;
                r1 = row;
            }
            return issue(&L.k, page, row);
        };
        auto values = [&]() -> bool {
            const int page = p0, row = r0;
            p0 = p1;
            r0 = r1;
            --held;
            return issue(&L.v, page, row);
        };
        if (!keys()) return;
        if (!WIDE && g.i1 - g.i0 > 1 && !keys()) return;
        for (int i = g.i0; i < g.i1; ++i) {
            if (!values()) return;
            if (i + (WIDE ? 1 : 2) < g.i1 && !keys()) return;
        }
    }
}

// ---------------------------------------------------------------- the MMA thread

template <int HD, bool WIDE>
__device__ __forceinline__ void mma_role(const Launch &L, Shared &s, uint32_t qbuf, uint32_t ring,
                                         Cursor cur, uint32_t tm) {
    using C = Cfg<HD>;
    constexpr int ROWS = WIDE ? 256 : 128;
    const AttnArgs &a = L.a;
    uint32_t pos = 0, seg = 0, np[2] = {0, 0}, nc[2] = {0, 0};
    Segment g;
    auto next_slot = [&](uint32_t &slot) -> bool {
        slot = pos % C::NS;
        const uint32_t round = pos / C::NS;
        ++pos;
        return wait_one(bar(s.b.full[slot]), round & 1, &s.dead);
    };
    auto scores = [&](int w, uint32_t slot) {
        const uint32_t q = qbuf + (WIDE ? w : (seg & 1)) * C::kTile, k = ring + slot * C::kTile;
        fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::kBox + (kk & 3) * 32;
            mma_ss(tm + w * 128, desc128(q + off, 16, 1024), desc128(k + off, 16, 1024),
                   idesc(128, false), kk > 0);
        }
        commit(bar(s.b.s_full[w]));
    };
    auto output = [&](int w, uint32_t slot, bool first) {
        const uint32_t v = ring + slot * C::kTile;
        fence_after();
#pragma unroll
        for (int kk = 0; kk < kKT / 16; ++kk)
            mma_ts(tm + C::kO + w * 128, tm + w * 128 + kP + kk * 8,
                   desc128(v + kk * 2048, C::kBox, 1024), idesc(HD, true), !first || kk > 0);
    };
    while (next_segment<ROWS, kKT>(a, cur, g)) {
        uint32_t ks;
        const int n = g.i1 - g.i0;
        if (!next_slot(ks)) return;
        if (WIDE) {
            for (int w = 0; w < 2; ++w) {
                if (!wait_one(bar(s.b.q_ready[w]), seg & 1, &s.dead)) return;
                scores(w, ks);
            }
            commit(bar(s.b.empty[ks]));
        } else {
            if (!wait_one(bar(s.b.q_ready[seg & 1]), (seg >> 1) & 1, &s.dead)) return;
            scores(0, ks);
            commit(bar(s.b.empty[ks]));
            if (n > 1) {
                if (!next_slot(ks)) return;
                scores(1, ks);
                commit(bar(s.b.empty[ks]));
            }
        }
        for (int i = 0; i < n; ++i) {
            uint32_t vs;
            if (!next_slot(vs)) return;
            const bool full = tile_full(a, g.span, tile_place<kKT>(g.span, g.i0 + i));
            if (WIDE) {
                if (!full && !wait_one(bar(s.b.clean[0]), nc[0]++ & 1, &s.dead)) return;
                const bool more = i + 1 < n;
                for (int w = 0; w < 2; ++w) {
                    if (!wait_one(bar(s.b.p_ready[w]), np[w]++ & 1, &s.dead)) return;
                    output(w, vs, i == 0);
                    if (w == 1) commit(bar(s.b.empty[vs]));
                    if (!more) {
                        commit(bar(s.b.o_full[w]));
                        continue;
                    }
                    if (w == 0 && !next_slot(ks)) return;
                    scores(w, ks);
                    if (w == 1) commit(bar(s.b.empty[ks]));
                }
            } else {
                const int w = i & 1;
                if (!full && !wait_one(bar(s.b.clean[w]), nc[w]++ & 1, &s.dead)) return;
                if (!wait_one(bar(s.b.p_ready[w]), np[w]++ & 1, &s.dead)) return;
                output(w, vs, i < 2);
                commit(bar(s.b.empty[vs]));
                if (i + 2 < n) {
                    if (!next_slot(ks)) return;
                    scores(w, ks);
                    commit(bar(s.b.empty[ks]));
                }
                if (i + 1 == n) commit(bar(s.b.o_full[0]));
            }
        }
        ++seg;
    }
}

// ---------------------------------------------------------------- the softmax warpgroups

// Adds the values that are not finite, at the places of the segment's masked
// tiles that the row at `place` sees, to output columns [col, col + 32).
__device__ __noinline__ void add_unbounded(const AttnArgs &a, const Segment &g, int place, int col,
                                           float *o) {
    for (int i = g.i0; i < g.i1; ++i) {
        const int j0 = tile_place<kKT>(g.span, i);
        if (tile_full(a, g.span, j0)) continue;
        for (int j = j0; j < j0 + kKT; ++j) {
            if (!unit_sees(a, g.span, j) || !row_sees(a, place, j)) continue;
            const int page = a.page_table[(long long)g.r * a.max_pages + (j >> a.page_shift)];
            if (page < 0 || page >= a.n_pages) continue;
            const __nv_bfloat16 *v =
                static_cast<const __nv_bfloat16 *>(a.v) + (long long)page * a.page_stride +
                (((long long)g.h << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * a.hd + col;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const float x = __bfloat162float(v[e]);
                if (!isfinite(x)) o[e] += x;
            }
        }
    }
}

template <int HD, bool WIDE>
__device__ __forceinline__ void softmax_role(const Launch &L, Shared &s, uint32_t qbuf, uint32_t ring,
                                             Cursor cur, Segment &g, bool &any, long long &x_end,
                                             uint32_t tm) {
    using C = Cfg<HD>;
    constexpr int ROWS = WIDE ? 256 : 128;
    constexpr int CR = HD / 8;  // 16-byte chunks of a row
    const AttnArgs &a = L.a;
    const int tid = threadIdx.x, w = tid >> 7, t = tid & 127;
    const uint32_t lane_base = (uint32_t)(t & ~31) << 16;
    const uint32_t ts = tm + w * 128 + lane_base, to = tm + C::kO + w * 128 + lane_base;

    // This thread's share of a segment's queries on their way to shared memory.
    auto load_queries = [&](const Segment &q, uint32_t seg) {
        const int first = WIDE ? w * 128 : w * 64, count = WIDE ? 128 : 64;
        const uint32_t dst = qbuf + (WIDE ? w : (seg & 1)) * C::kTile;
        const int rows = q.req.T * a.G - q.qt * ROWS;
        for (int x = t; x < count * CR; x += 128) {
            const int i = first + x / CR, c = x % CR, r = i & 127;
            const int row = q.qt * ROWS + i, tok = row / a.G;
            const uint32_t at = dst + (c >> 3) * C::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q);
            const bool has = i < rows;
            if (has) src += (q.req.row0 + tok) * a.q_stride + (q.h * a.G + row % a.G) * HD + c * 8;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(at), "l"(src),
                         "r"(has ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    auto queries_ready = [&](uint32_t seg) {
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        fence_async();
        arrive(bar(s.b.q_ready[WIDE ? w : (seg & 1)]));
    };

    uint32_t seg = 0, base_pos = 0, n_s = 0;
    Segment gn;
    bool more = next_segment<ROWS, kKT>(a, cur, gn);
    if (more) {
        load_queries(gn, 0);
        queries_ready(0);
    }
    while (more) {
        g = gn;
        any = true;
        x_end = cur.x;
        Cursor ahead = cur;
        more = next_segment<ROWS, kKT>(a, ahead, gn);
        const int n = g.i1 - g.i0;
        const TileSpan sp = g.span;
        const int row = g.qt * ROWS + (WIDE ? w * 128 : 0) + t;
        const bool has = row < g.req.T * a.G;
        const int place = g.req.ctx + row / a.G;
        bool q_pending = false;
        if (!WIDE && more) {  // the other buffer is free: the last segment is done with it
            load_queries(gn, seg + 1);
            q_pending = true;
        }
        float m = -INFINITY, l = 0.f;
        for (int i = WIDE ? 0 : w; i < n; i += WIDE ? 1 : 2) {
            const int j0 = tile_place<kKT>(sp, g.i0 + i);
            const bool full = tile_full(a, sp, j0);
            if (!wait(bar(s.b.s_full[w]), n_s++ & 1, &s.dead)) return;
            fence_after();
            if (WIDE && i + 1 == n && more) {  // this warpgroup's queries are no longer read
                load_queries(gn, seg + 1);
                q_pending = true;
            }
            if (!full) {
                // Clear what must not be seen from the value tile.
                const uint32_t pos = base_pos + (WIDE ? 2 * i + 1 : min(n, i + 2) + i);
                const uint32_t slot = pos % C::NS, vt = ring + slot * C::kTile;
                if (!wait(bar(s.b.full[slot]), (pos / C::NS) & 1, &s.dead)) return;
                const int r = WIDE ? w * 64 + (t >> 1) : t;
                const int c0 = WIDE ? (t & 1) * (CR / 2) : 0, c1 = c0 + (WIDE ? CR / 2 : CR);
                const bool seen = unit_sees(a, sp, j0 + r);
                for (int c = c0; c < c1; ++c) {
                    const uint32_t at = vt + (c >> 3) * C::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    uint32_t x[4] = {0, 0, 0, 0};
                    bool write = !seen;
                    if (seen) {
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                     : "r"(at)
                                     : "memory");
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((x[e] & 0x7F80u) == 0x7F80u) x[e] &= 0xFFFF0000u, write = true;
                            if ((x[e] & 0x7F800000u) == 0x7F800000u) x[e] &= 0xFFFFu, write = true;
                        }
                        if (write) s.poison[seg & 3] = (int)seg;
                    }
                    if (write)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]),
                                     "r"(x[1]), "r"(x[2]), "r"(x[3])
                                     : "memory");
                }
                fence_async();
                arrive(bar(s.b.clean[WIDE ? 0 : w]));
            }
            // The scores, half a row at a time: the second half stays in registers from
            // the maximum to the weights, the first is read twice.
            uint32_t x[64];
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const int hi = place - j0, lo = a.window ? hi - a.window : -1, sk = a.sinks - j0;
            auto scores = [&](int half) {
                tmem_ld32(ts + half * 64, x);
                tmem_ld32(ts + half * 64 + 32, x + 32);
                wait_ld();
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        const int c = half * 64 + e;
                        if (c > hi || (c <= lo && c >= sk)) x[e] = 0xff800000u;  // -inf
                    }
                }
            };
            auto maximum = [&]() {
#pragma unroll
                for (int e = 0; e < 64; ++e) top4[e & 3] = fmaxf(top4[e & 3], __uint_as_float(x[e]));
            };
            scores(0);
            maximum();
            scores(1);
            maximum();
            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * a.scale_log2;
            if (__any_sync(0xffffffffu, top > m + kLazy)) {
                const float mn = fmaxf(m, top);
                const float keep = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
                m = mn;
                l *= keep;
                if (i >= (WIDE ? 1 : 2)) {
#pragma unroll 1
                    for (int q = 0; q < HD / 32; ++q) {
                        uint32_t y[32];
                        tmem_ld32(to + 32 * q, y);
                        wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * keep);
                        tmem_st32(to + 32 * q, y);
                    }
                }
            }
            const float off = m == -INFINITY ? 0.f : -m;
            float sum4[4] = {0.f, 0.f, 0.f, 0.f};
            auto weights = [&](int half) {
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float y0 = exp2_fast(fmaf(__uint_as_float(x[e]), a.scale_log2, off));
                    const float y1 = exp2_fast(fmaf(__uint_as_float(x[e + 1]), a.scale_log2, off));
                    sum4[e & 2] += y0;
                    sum4[(e & 2) + 1] += y1;
                    x[e / 2] = pack_bf16(y0, y1);
                }
                tmem_st32(ts + kP + half * 32, x);  // over scores that are not needed any more
            };
            weights(1);
            scores(0);
            weights(0);
            l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
            wait_st();
            fence_before();
            arrive(bar(s.b.p_ready[w]));
            if (q_pending) {
                queries_ready(seg + 1);
                q_pending = false;
            }
        }
        if (q_pending) queries_ready(seg + 1);

        // The end of the segment.
        if (!wait(bar(s.b.o_full[WIDE ? w : 0]), seg & 1, &s.dead)) return;
        fence_after();
        const bool poisoned = *(volatile int *)&s.poison[seg & 3] == (int)seg;
        const bool whole = g.i0 == 0 && g.i1 == sp.n;
        float f0 = 1.f, f1 = 0.f;
        int c0 = 0, c1 = HD;
        uint32_t ta = to, tb = to;
        if (!WIDE) {
            // Join: each warpgroup writes half of the columns of both outputs.
            s.m[w][t] = m;
            s.l[w][t] = l;
            arrive(bar(s.b.joined));
            if (!wait(bar(s.b.joined), 0, &s.dead)) return;
            const float m0 = s.m[0][t], m1 = s.m[1][t];
            m = fmaxf(m0, m1);
            const float base = m == -INFINITY ? 0.f : m;
            f0 = exp2_fast(m0 - base);
            f1 = exp2_fast(m1 - base);
            l = s.l[0][t] * f0 + s.l[1][t] * f1;
            c0 = w * (HD / 2);
            c1 = c0 + HD / 2;
            ta = tm + C::kO + lane_base;
            tb = ta + 128;
        }
        const long long at = (long long)(g.req.row0 + row / a.G) * a.Hq + g.h * a.G + row % a.G;
        const float inv = 1.f / l;
        float *part = a.part + (long long)part_slot(blockIdx.x, g) * ROWS * (HD + 2);
        const int prow = WIDE ? w * 128 + t : t;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
            uint32_t y[32];
            float o[32];
            tmem_ld32(ta + c, y);
            wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(y[e]) * f0;
            if (!WIDE && n > 1) {  // one tile: the second warpgroup had none
                tmem_ld32(tb + c, y);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(__uint_as_float(y[e]), f1, o[e]);
            }
            if (poisoned) add_unbounded(a, g, place, c, o);
            if (!has) continue;
            if (whole) {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * HD + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dst[e] = make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv),
                                        pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                        pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                        pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
            } else {
                float4 *dst = reinterpret_cast<float4 *>(part + (long long)prow * HD + c);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
        }
        if (has && (WIDE || w == 0)) {
            if (whole) {
                if (a.lse) a.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
            } else {
                part[ROWS * HD + prow] = m;
                part[ROWS * HD + ROWS + prow] = l;
            }
        }
        if (!WIDE) {  // both outputs have been read: either may be written again
            fence_before();
            arrive(bar(s.b.joined));
            if (!wait(bar(s.b.joined), 1, &s.dead)) return;
            fence_after();
        }
        base_pos += 2 * n;
        ++seg;
        cur = ahead;
    }
}

template <int HD, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ Launch L) {
    using C = Cfg<HD>;
    constexpr int ROWS = WIDE ? 256 : 128;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char raw[];  // the tiles first: whole swizzle atoms
    Shared &s = *reinterpret_cast<Shared *>(raw + C::kTiles);
    const uint32_t base = smem_addr(raw);
    const uint32_t qbuf = base, ring = base + 2 * C::kTile;
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(bar(s.b.full[i]), 1);
            mbar_init(bar(s.b.empty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(s.b.s_full[w]), 1);
            mbar_init(bar(s.b.p_ready[w]), 128);
            mbar_init(bar(s.b.o_full[w]), 1);
            mbar_init(bar(s.b.q_ready[w]), WIDE ? 128 : 256);
            mbar_init(bar(s.b.clean[w]), WIDE ? 256 : 128);
        }
        mbar_init(bar(s.b.joined), 256);
        mbar_init(bar(s.b.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s.dead = 0;
        for (int i = 0; i < 4; ++i) s.poison[i] = -1;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&L.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&L.v)) : "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                         smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    Cursor cur = make_plan<kThreads, ROWS, kKT, 1>(L.a, blockIdx.x, gridDim.x, &s.plan,
                                                   blockIdx.x == 0);
    fence_after();
    const uint32_t tm = *(volatile uint32_t *)&s.tmem;

    if (warp < 8) {
        Segment g;
        bool any = false;
        long long x_end = 0;
        softmax_role<HD, WIDE>(L, s, qbuf, ring, cur, g, any, x_end, tm);
        if (tid == 0) write_desc(L.a, blockIdx.x, g, any, x_end, s.plan.total, s.plan.workers);
    } else {
        if (warp == 8) {
            uint32_t issued = 0;
            load_role<HD, WIDE>(L, s, ring, cur, tid & 31, issued);
            // Every copy has landed before the block ends (the roles waited for them
            // unless one gave up).
            for (uint32_t p = issued > C::NS ? issued - C::NS : 0; p < issued; ++p)
                wait_parity(bar(s.b.full[p % C::NS]), (p / C::NS) & 1);
        } else if (tid == 9 * 32) {
            mma_role<HD, WIDE>(L, s, qbuf, ring, cur, tm);
            commit(bar(s.b.drain));
            wait_parity(bar(s.b.drain), 0);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (tid == 0 && s.dead && L.a.dev_err) atomicOr(L.a.dev_err, GDN_DEVERR_TIMEOUT);
    if (warp == 9) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tm) : "memory");
    }
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Pages [n_pages][kv_heads][page][hd]; boxes of 64 columns by up to 128 places of one
// head of one page.  Pages past the end read as zeros.
bool encode_pages(CUtensorMap *map, const AttnArgs &a, const void *base) {
    const cuuint64_t page = 1ull << a.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)a.hd, page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.hd * 2, page * a.hd * 2,
                                   (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)(page < kKT ? page : kKT), 1, 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                     strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, bool WIDE>
cudaError_t launch_tc(const AttnArgs &a, cudaStream_t stream) {
    Launch L;
    L.a = a;
    if (!encoder() || !encode_pages(&L.k, a, a.k) || !encode_pages(&L.v, a, a.v))
        return cudaErrorInvalidValue;
    constexpr int smem = Cfg<HD>::kTiles + (int)sizeof(Shared);
    static_assert(smem <= 232448, "227 KB of shared memory a block");
    const cudaError_t e = cudaFuncSetAttribute(
        attn_tc_kernel<HD, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnTcWorkers);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc_kernel<HD, WIDE>, L);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, bool wide, cudaStream_t stream) {
    if (a.hd == 64) return wide ? launch_tc<64, true>(a, stream) : launch_tc<64, false>(a, stream);
    return wide ? launch_tc<128, true>(a, stream) : launch_tc<128, false>(a, stream);
}

}  // namespace gdn
