// Attention over a paged cache on the tensor cores (tcgen05): drafts of many
// query rows a key head, and prompt chunks (bf16, heads of 64 and 128).
//
// A lane-parallel TMA warp streams keys and values, page by page, into a ring in
// shared memory (128-byte swizzle; a page that no row needs, or that does not exist, is
// asked for past the tensor's end and reads as zeros without traffic).  One thread
// issues the products: S = Q K^T with both operands in shared memory, O += P V with
// the weights P in tensor memory.  A warpgroup does the softmax of 128 rows, a thread a
// row, with its S and O in tensor memory.
//
//   Prompt chunks: two warpgroups, 256 rows of a unit, one block an SM, tiles of 128
//     places that both use.  The tensor cores work for one warpgroup while the other is
//     between its products.  Bound by the tensor cores: 2 * 128^2 * HD * 2 flops a
//     tile and warpgroup.
//   Drafts, up to 128 rows a key head: one warpgroup, tiles of 16 KB, two blocks an
//     SM, so that one streams while the other ends a unit.  Bound by the cache's bytes;
//     rows that are not there cost tensor time that the stream leaves over.
//
// Measured (bf16): two requests' prompt chunks of 4001 rows over 6007 places, 32 heads
// on 8 key heads of 128: 665 to 740 us by the clocks that the power leaves, 1.42 to 1.58
// PFLOP/s of visible products, tensor pipe 68% busy
// (the tensor cores wait while a warpgroup hands its weights over).  8000 rows behind a
// window of 512, heads of 64: 162 us; a unit has six tiles, so its start and end and the
// masked tiles are most of it.  64 requests' 16 drafts over up to 4000 places: 0.67 GB in 125 us,
// 5.4 TB/s.  128 requests' up to 16 drafts behind a window of 1024: 75 us, 290 MB; the
// units are short.  16 drafts over 130001 places, heads of 64: 61 us, 4.4 TB/s; its 38
// partials to each of eight units are joined by a second launch.
//
// A row's maximum is replaced, and its output rescaled in tensor memory, only
// when it has grown by more than 2^8 (kLazy): the weights then stay below 2^8,
// which their float32 sums hold as exactly.  The weights are rounded to bf16 for
// the second product (its operands have one type); their total is summed
// before the rounding.
//
// Places that no row sees, and values that are not finite where some rows must
// not see them, would still reach the output as 0 * NaN.  In the tiles where
// any row's mask hides something (the ends of a unit) a warp therefore clears them
// from the value tile first; the rows that do see such a value get it
// added at the end (add_unbounded).
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_launch.h"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kSegs = 4;       // segments known ahead
constexpr float kLazy = 8.f;
constexpr int kGroup = 8;      // partials joined at a time
static_assert(kGroup * kGroup * kGroup >= kAttnWorkers && kAttnLevels == 3, "levels of groups");

// NWG softmax warpgroups, then the TMA, MMA, segment and clearing warps.
template <int HD, int NWG>
struct Cfg {
    static constexpr int KT = NWG == 2 || HD == 64 ? 128 : 64;  // places of a tile
    static constexpr int ROWS = 128 * NWG;             // rows of a unit
    // A unit's start and end, in tiles, and the places of the line that a worker has at least.
    // With 2 tiles the drafts and prompts measured stay within 3%; with 1 or 12 heads of 64
    // lose 14% (3829 rows: 353 us, 403 and 401).  With 10, 16 or 24 places the smallest
    // calls lose 3 to 14 us (13 requests of up to 32 rows over 640 places: 16 us, 19, 23 and 27).
    static constexpr int EXTRA = 4, kMin = 6;
    static constexpr int kThreads = 128 * NWG + 128;
    static constexpr int kBlocks = NWG == 2 ? 1 : 2;   // an SM
    static constexpr int kTile = KT * HD * 2;          // bytes of a key (value) tile
    static constexpr int kBox = KT * 128;              // bytes of 64 of its columns
    static constexpr int kQTile = 128 * HD * 2, kQBox = 128 * 128;
    static constexpr int NS = HD == 128 ? 5 : NWG == 2 ? 12 : 6;  // ring slots
    static constexpr int kTiles = NWG * kQTile + NS * kTile;
    // Columns of tensor memory.  Two weights are a column; P_w lies over the second half of
    // S_w where the columns are all needed.
    static constexpr uint32_t kCols = NWG == 2 ? 512 : 256;
    static constexpr uint32_t kP = 64, kO = NWG == 2 ? 256 : 128;
};

constexpr int kCleans = 8;  // value tiles between the warp that clears them and their products

struct Bars {
    unsigned long long full[12], empty[12];
    unsigned long long s_full[2], p_ready[2], o_full, q_ready[2], q_free, clean[kCleans], staged, drain, joined[2];
    unsigned long long seg_full[kSegs], seg_empty[kSegs];
};

struct Shared {
    Bars b;
    PlanScratch plan;
    uint32_t tmem;
    int dead;          // a wait gave up: every role leaves
    int poison[4];     // segment (mod 4) whose hidden places hold values that are not finite
    int join[2];       // whether a warpgroup is to join a group of partials
    Segment seg[kSegs];  // r = -1: no more
};

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                       int c3, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(b)
        : "memory");
}

// Places of a TMA box: a page, or a tile's worth of one.
__host__ __device__ __forceinline__ int box_rows(const AttnArgs &a, int kt) {
    return 1 << a.page_shift < kt ? 1 << a.page_shift : kt;
}

struct Launch {
    AttnArgs a;
    CUtensorMap k, v, q;
    int q_tma;  // the queries come by TMA too: a power of two of heads a group, up to 128
};

// ---------------------------------------------------------------- the segment thread

// Works out the worker's segments ahead of the roles that use them (each takes loads that
// wait on one another).
template <typename C>
__device__ __forceinline__ void segment_role(const AttnArgs &a, Shared &s, Cursor cur) {
    Ring<kSegs> ring;
    for (;;) {
        Segment g;
        const bool more = next_segment<C::ROWS, C::KT, C::EXTRA>(a, box_rows(a, C::KT), cur, g);
        if (!more) g.r = -1;
        if (!wait_one(bar(s.b.seg_empty[ring.slot]), ring.parity ^ 1, &s.dead)) return;
        s.seg[ring.slot] = g;
        arrive(bar(s.b.seg_full[ring.slot]));
        if (!more) return;
        ring.next();
    }
}

// A warp's view of the segments.
struct SegReader {
    Ring<kSegs> ring;
    // The next segment, in shared memory until it is released; NULL after the last.
    __device__ __forceinline__ const Segment *peek(Shared &s) {
        if (!wait(bar(s.b.seg_full[ring.slot]), ring.parity, &s.dead)) return nullptr;
        return s.seg[ring.slot].r >= 0 ? &s.seg[ring.slot] : nullptr;
    }
    __device__ __forceinline__ bool next(Shared &s, Segment &g) {  // a copy
        const Segment *p = peek(s);
        if (!p) return false;
        g = *p;
        arrive_warp(bar(s.b.seg_empty[ring.slot]));
        ring.next();
        return true;
    }
};

// ---------------------------------------------------------------- the TMA warp

template <int HD, int NWG>
__device__ __forceinline__ void load_role(const Launch &L, Shared &s, uint32_t qbuf, uint32_t ring, int lane,
                                          uint32_t &issued, uint32_t &seg) {
    using C = Cfg<HD, NWG>;
    const AttnArgs &a = L.a;
    const int rows_box = box_rows(a, C::KT);
    const int boxes = C::KT / rows_box;
    Ring<C::NS> at;
    SegReader segs;
    Segment g, gn;
    // This lane's page of tile i of a segment: its row and number, or n_pages (nothing
    // needed, or no page).
    auto page_of = [&](const Segment &q, int i, int &row) -> int {
        const int v = i * C::KT + lane * rows_box, j = place_of(q.span, v);
        row = j & ((1 << a.page_shift) - 1);
        if (lane >= boxes || !some_see(a, q.span, v, v + rows_box - 1)) return (int)a.n_pages;
        const int page = a.page_table[(long long)q.r * a.max_pages + (j >> a.page_shift)];
        if (page >= 0 && page < a.n_pages) return page;
        if (a.dev_err) atomicOr(a.dev_err, GDN_DEVERR_PAGE);
        return (int)a.n_pages;
    };
    auto issue = [&](const CUtensorMap *map, int page, int row) -> bool {
        if (!wait(bar(s.b.empty[at.slot]), at.parity ^ 1, &s.dead)) return false;
        const uint32_t f = bar(s.b.full[at.slot]);
        if (lane == 0) arrive_expect(f, C::kTile);
        __syncwarp();
        if (lane < boxes) {
            const uint32_t dst = ring + at.slot * C::kTile + lane * rows_box * 128;
#pragma unroll
            for (int h = 0; h < HD / 64; ++h)
                tma_4d(dst + h * C::kBox, map, 64 * h, row, g.h, page, f);
        }
        at.next();
        ++issued;
        return true;
    };
    // The queries of segment `seg`, 128 rows of (token, head of the group) a warpgroup.  Rows
    // past the request's are other tokens', or zeros: their results are not used.
    auto queries = [&]() -> bool {
        // the last segment has computed its last scores
        if (seg > 0 && !wait(bar(s.b.q_free), (seg - 1) & 1, &s.dead)) return false;
        if (lane == 0) {
#pragma unroll
            for (int w = 0; w < NWG; ++w) {
                const uint32_t r = bar(s.b.q_ready[w]), dst = qbuf + w * C::kQTile;
                const int token = g.req.row0 + div_group(a, g.qt * C::ROWS + w * 128);
                arrive_expect(r, C::kQTile);
#pragma unroll
                for (int h = 0; h < HD / 64; ++h)
                    tma_4d(dst + h * C::kQBox, &L.q, 64 * h, 0, g.h, token, r);
            }
        }
        __syncwarp();
        ++seg;
        return true;
    };
    // Pages are looked up a tile ahead, across segments too.
    int row_n = 0, next = 0;
    bool more = segs.next(s, g);
    if (more) next = page_of(g, g.i0, row_n);
    while (more) {
        int ik = g.i0, page = 0, row = 0;  // of the tile whose values are to come
        more = segs.next(s, gn);
        auto keys = [&]() -> bool {
            page = next;
            row = row_n;
            if (++ik < g.i1)
                next = page_of(g, ik, row_n);
            else if (more)
                next = page_of(gn, gn.i0, row_n);
            return issue(&L.k, page, row);
        };
        if (!keys()) return;
        if (L.q_tma && !queries()) return;
        for (int i = g.i0; i < g.i1; ++i) {
            if (!issue(&L.v, page, row)) return;
            if (i + 1 < g.i1 && !keys()) return;
        }
        g = gn;
    }
}

// ---------------------------------------------------------------- the MMA warp

template <int HD, int NWG>
__device__ __forceinline__ void mma_role(Shared &s, uint32_t qbuf, uint32_t ring,
                                         uint32_t tm) {
    using C = Cfg<HD, NWG>;
    Ring<C::NS> at;
    SegReader segs;
    const uint32_t lead = elect();
    uint32_t seg = 0, tiles = 0, staged = 0;  // so far
    Ring<kCleans> clean;
    uint32_t held = 0;      // ring slot the softmax warpgroups stage their output in
    bool holding = false;
    Segment g;
    tm = __shfl_sync(0xffffffffu, tm, 0);
    const uint32_t q_lo = desc_lo(qbuf, 16), k_lo = desc_lo(ring, 16), v_lo = desc_lo(ring, C::kBox);
    auto next_slot = [&](uint32_t &slot) -> bool {
        slot = at.slot;
        const bool ok = wait(bar(s.b.full[at.slot]), at.parity, &s.dead);
        at.next();
        return ok;
    };
    auto next_values = [&](uint32_t &slot) -> bool {  // there, and cleared of what must not be seen
        slot = at.slot;
        at.next();
        const bool ok = wait(bar(s.b.clean[clean.slot]), clean.parity, &s.dead);
        clean.next();
        return ok;
    };
    auto scores = [&](int w, uint32_t slot) {
        const uint32_t q = q_lo + w * (C::kQTile >> 4), k = k_lo + slot * (C::kTile >> 4);
        fence_after();
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
            mma_ss(lead, tm + w * 128, q + (((kk >> 2) * C::kQBox + (kk & 3) * 32) >> 4),
                   k + (((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4), idesc(C::KT, false), kk > 0);
        commit(lead, bar(s.b.s_full[w]));
    };
    auto output = [&](int w, uint32_t slot, bool first) -> bool {
        const uint32_t v = v_lo + slot * (C::kTile >> 4);
        const uint32_t acc = first ? 0u : 1u;
        if (!wait(bar(s.b.p_ready[w]), tiles & 1, &s.dead)) return false;
        fence_after();
#pragma unroll
        for (int kk = 0; kk < C::KT / 16; ++kk)
            mma_ts(lead, tm + C::kO + w * 128, tm + w * 128 + C::kP + kk * 8, v + kk * (2048 >> 4),
                   idesc(HD, true), kk > 0 ? 1u : acc);
        return true;
    };
    // The slot of the last segment's last values goes back to the ring when the warpgroups
    // have written their output from it.
    auto give_back = [&]() -> bool {
        if (!holding) return true;
        if (!wait(bar(s.b.staged), staged++ & 1, &s.dead)) return false;
        if (lead) arrive(bar(s.b.empty[held]));
        __syncwarp();
        holding = false;
        return true;
    };
    while (segs.next(s, g)) {
        uint32_t ks, vs = 0;
        const int n = __shfl_sync(0xffffffffu, g.i1 - g.i0, 0);
        if (!next_slot(ks)) return;
#pragma unroll
        for (int w = 0; w < NWG; ++w) {
            if (!wait(bar(s.b.q_ready[w]), seg & 1, &s.dead)) return;
            scores(w, ks);
        }
        commit(lead, bar(s.b.empty[ks]));
        if (n == 1) commit(lead, bar(s.b.q_free));
        if (!give_back()) return;
        for (int i = 0; i < n; ++i, ++tiles) {
            if (!next_values(vs)) return;
#pragma unroll
            for (int w = 0; w < NWG; ++w) {
                if (!output(w, vs, i == 0)) return;
                const bool last = w == NWG - 1;
                if (i + 1 < n) {
                    if (w == 0 && !next_slot(ks)) return;
                    if (last) commit(lead, bar(s.b.empty[vs]));
                    scores(w, ks);
                    if (last) commit(lead, bar(s.b.empty[ks]));
                    if (last && i + 2 == n) commit(lead, bar(s.b.q_free));
                } else if (last) {  // all at once: the outputs are staged over the values
                    commit(lead, bar(s.b.o_full));
                }
            }
        }
        held = vs;
        holding = true;
        ++seg;
    }
}

// ---------------------------------------------------------------- the clearing warp

// Hands each value tile on to its products.  It takes part in the release of every ring
// slot, keys too: a wait on a barrier's parity is only right for one that has seen
// the phase before, so no slot may come round twice without it.  In value tiles that
// hold places hidden from some row it first clears the places that no row sees, and
// the elements that are not finite where only some rows see them.
template <int HD, int NWG>
__device__ __forceinline__ void clear_role(const Launch &L, Shared &s, uint32_t ring, int lane) {
    using C = Cfg<HD, NWG>;
    constexpr int CR = HD / 8;  // 16-byte chunks of a row
    const AttnArgs &a = L.a;
    Ring<C::NS> at;
    Ring<kCleans> clean;
    SegReader segs;
    uint32_t seg = 0;
    Segment g;
    while (segs.next(s, g)) {
        const int n = g.i1 - g.i0;
        auto keys = [&]() -> bool {
            if (!wait(bar(s.b.full[at.slot]), at.parity, &s.dead)) return false;
            arrive_warp(bar(s.b.empty[at.slot]));
            at.next();
            return true;
        };
        if (!keys()) return;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (!wait(bar(s.b.full[at.slot]), at.parity, &s.dead)) return;
            const int v0 = (g.i0 + i) * C::KT;
            if (!all_see(a, g.span, v0, v0 + C::KT - 1)) {
                const uint32_t vt = ring + at.slot * C::kTile;
#pragma unroll 1
                for (int r = lane; r < C::KT; r += 32) {
                    const int v = v0 + r;
                    if (all_see(a, g.span, v, v)) continue;
                    auto chunk = [&](int c) {
                        return vt + (c >> 3) * C::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                    };
                    if (!some_see(a, g.span, v, v)) {
#pragma unroll
                        for (int c = 0; c < CR; ++c)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(chunk(c)),
                                         "r"(0)
                                         : "memory");
                        continue;
                    }
                    // Not finite: the exponent is all ones.
                    uint32_t odd = 0;
#pragma unroll
                    for (int c = 0; c < CR; ++c) {
                        uint32_t x[4];
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                     : "r"(chunk(c))
                                     : "memory");
#pragma unroll
                        for (int e = 0; e < 4; ++e) odd |= (x[e] & 0x7F807F80u) + 0x00800080u;
                    }
                    if (odd & 0x80008000u) {
                        s.poison[seg & 3] = (int)seg;
#pragma unroll 1
                        for (int c = 0; c < CR * 4; ++c) {
                            uint32_t x;
                            const uint32_t to = chunk(c >> 2) + (c & 3) * 4;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(to) : "memory");
                            if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
                            if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
                            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
                        }
                    }
                }
                fence_async();
            }
            arrive_warp(bar(s.b.clean[clean.slot]));
            arrive_warp(bar(s.b.empty[at.slot]));
            clean.next();
            at.next();
            if (i + 1 < n && !keys()) return;
        }
        ++seg;
    }
}

// ---------------------------------------------------------------- the softmax warpgroups

// Adds the values that are not finite, at the places of the segment's masked
// tiles that the row at number `own` sees, to output columns [col, col + 32).
__device__ __noinline__ void add_unbounded(const AttnArgs &a, const Segment &g, int kt, int own, int col,
                                           float *o) {
    for (int i = g.i0; i < g.i1; ++i) {
        if (all_see(a, g.span, i * kt, i * kt + kt - 1)) continue;
        for (int v = i * kt; v < (i + 1) * kt; ++v) {
            if (!some_see(a, g.span, v, v) || all_see(a, g.span, v, v) || !row_sees(a, g.span, own, v))
                continue;
            const int j = place_of(g.span, v);
            const int page = a.page_table[(long long)g.r * a.max_pages + (j >> a.page_shift)];
            if (page < 0 || page >= a.n_pages) continue;
            const __nv_bfloat16 *x =
                static_cast<const __nv_bfloat16 *>(a.v) + (long long)page * a.page_stride +
                (((long long)g.h << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * a.hd + col;
            for (int e = 0; e < 32; ++e) {
                const float f = __bfloat162float(x[e]);
                if (!isfinite(f)) o[e] += f;
            }
        }
    }
}

template <int HD, int NWG>
__device__ __forceinline__ void softmax_role(const Launch &L, Shared &s, uint32_t qbuf, uint32_t ring,
                                             uint32_t tm, const Cursor &plan) {
    using C = Cfg<HD, NWG>;
    constexpr int ROWS = C::ROWS, KT = C::KT;
    constexpr int CR = HD / 8;  // 16-byte chunks of a row
    const AttnArgs &a = L.a;
    const int tid = threadIdx.x, w = tid >> 7, t = tid & 127, lane = tid & 31;
    const uint32_t lane_base = (uint32_t)(t & ~31) << 16;
    const uint32_t ts = tm + w * 128 + lane_base, to = tm + C::kO + w * 128 + lane_base;
    SegReader segs;

    // This thread's share of its warpgroup's queries on their way to shared memory (where TMA
    // does not bring them): sixteen (eight) threads a row, rows 128 / CR apart.
    auto load_queries = [&](const Segment &q) {
        const int rows = q.req.T * a.G - q.qt * ROWS - w * 128;
        const uint32_t dst = qbuf + w * C::kQTile;
        const int c = t % CR;
        const __nv_bfloat16 *base = static_cast<const __nv_bfloat16 *>(a.q) + q.h * a.G * HD + c * 8;
#pragma unroll 4
        for (int r = t / CR; r < 128; r += 128 / CR) {
            const int row = q.qt * ROWS + w * 128 + r, tok = div_group(a, row);
            const uint32_t at = dst + (c >> 3) * C::kQBox + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            const bool has = r < rows;
            const __nv_bfloat16 *src =
                base + (has ? (q.req.row0 + tok) * a.q_stride + (row - tok * a.G) * HD : 0);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(at), "l"(src),
                         "r"(has ? 16 : 0)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    auto queries_ready = [&]() {
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        fence_async();
        arrive_warp(bar(s.b.q_ready[w]));
    };

    uint32_t seg = 0, n_s = 0;
    uint32_t base_slot = 0;  // ring slot of the segment's first tile
    if (!a.count && tid == 0)  // nothing left unfinished yet
        write_desc(a, blockIdx.x, s.seg[0], false, 0, 1, 1);
    const Segment *ahead = segs.peek(s);
    if (ahead && !L.q_tma) {
        load_queries(*ahead);
        queries_ready();
    }
    while (ahead) {
        const Segment &g = *ahead;
        const uint32_t seg_slot = segs.ring.slot;
        segs.ring.next();
        ahead = segs.peek(s);
        const int n = g.i1 - g.i0;
        const TileSpan sp = g.span;
        const int row = g.qt * ROWS + w * 128 + t;
        const int own = g.req.ctx + div_group(a, row) - sp.shift;  // its place, as numbered in the span
        float m = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const int v0 = (g.i0 + i) * KT;
            const bool full = all_see(a, sp, v0, v0 + KT - 1);
            if (!wait(bar(s.b.s_full[w]), n_s++ & 1, &s.dead)) return;
            fence_after();
            if (i + 1 == n && ahead && !L.q_tma) {  // this warpgroup's queries are no longer read
                load_queries(*ahead);
            }
            uint32_t x[64];
            uint32_t mask[KT / 32];  // of the tile's places, those that the row sees
            if (!full) {
                // number v0 + 32 q + e is bit e of mask[q]
                const int hi = own - v0, lo = a.window ? hi - a.window : -1, sk = sp.sinks - v0;
#pragma unroll
                for (int q = 0; q < KT / 32; ++q) {
                    // bits below x, of 32
                    auto below = [](int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; };
                    mask[q] = below(hi + 1 - 32 * q) &
                              (~below(lo + 1 - 32 * q) | below(sk - 32 * q));
                }
            }
            // The scores, 64 of a row at a time.  Of 128 the second half stays in registers from
            // the maximum to the weights, and the first is read twice.
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            auto scores = [&](int half, bool masked) {
                tmem_ld32(ts + half * 64, x);
                tmem_ld32(ts + half * 64 + 32, x + 32);
                wait_ld();
                if (masked) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t seen = mask[half * 2 + q];
                        if (__all_sync(0xffffffffu, seen == ~0u)) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(seen & (1u << e))) x[32 * q + e] = 0xff800000u;  // -inf
                    }
                }
            };
            auto maximum = [&]() {
#pragma unroll
                for (int e = 0; e < 64; e += 2)
                    top4[(e >> 1) & 3] = max3(top4[(e >> 1) & 3], __uint_as_float(x[e]),
                                              __uint_as_float(x[e + 1]));
            };
            scores(0, !full);
            maximum();
            if (KT == 128) {
                if (!full) {  // masked once: the second reading finds it so
                    tmem_st32(ts, x);
                    tmem_st32(ts + 32, x + 32);
                    wait_st();
                }
                scores(1, !full);
                maximum();
            }
            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * a.scale_log2;
            if (__any_sync(0xffffffffu, top > m + kLazy)) {
                const float mn = fmaxf(m, top);
                const float keep = mn == -INFINITY ? 1.f : exp2_fast(m - mn);
                m = mn;
                l *= keep;
                if (i > 0) {
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
            const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), off2 = make_float2(off, off);
            float2 sum[2] = {};
            auto weights = [&](int half) {
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                    scale2, off2);
                    y.x = exp2_fast(y.x);
                    y.y = exp2_fast(y.y);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], y);
                    x[e / 2] = pack_bf16(y.x, y.y);
                }
                tmem_st32(ts + C::kP + half * 32, x);  // over scores that are not needed any more
            };
            if (KT == 128) {
                weights(1);
                scores(0, false);
            }
            weights(0);
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            wait_st();
            fence_before();
            arrive_warp(bar(s.b.p_ready[w]));
            if (i + 1 == n && ahead && !L.q_tma) queries_ready();
        }

        // The end of the segment.
        if (!wait(bar(s.b.o_full), seg & 1, &s.dead)) return;
        fence_after();
        const bool poisoned = *(volatile int *)&s.poison[seg & 3] == (int)seg;
        const bool whole = g.i0 == 0 && g.i1 == sp.n;
        const int rows = g.req.T * a.G;
        const float inv = whole ? 1.f / l : 1.f;
        float *part = a.part + (long long)part_slot(blockIdx.x, g) * ROWS * (HD + 2);
        const int prow = w * 128 + t;
        // A finished unit's rows go through the slot of its last value tile, whose products
        // are done, so that whole lines are written: a warp's 32 rows, half of the columns
        // at a time.
        constexpr int NC = HD / 2, CPR = NC / 8;  // columns, chunks of a row
        // The segment's 2 n tiles took ring slots from base_slot on, this one the last.
        const uint32_t stage = ring + (base_slot + 2 * n - 1) % C::NS * C::kTile +
                               (tid >> 5) * (C::kTile / (4 * NWG));
        auto stage_at = [&](int r, int c) {
            return stage + r * NC * 2 + ((c ^ (CPR == 8 ? r & 7 : (r >> 1) & 3)) << 4);
        };
#pragma unroll 1
        for (int rd = 0; rd < 2; ++rd) {
#pragma unroll 1
            for (int c = 0; c < NC; c += 32) {
                const int col = rd * NC + c;
                uint32_t y[32];
                tmem_ld32(to + col, y);
                wait_ld();
                if (poisoned) {
                    float o[32];
                    for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(y[e]);
                    add_unbounded(a, g, C::KT, own, col, o);
                    for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(o[e]);
                }
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = pack_bf16(__uint_as_float(y[8 * e + 2 * k]) * inv,
                                             __uint_as_float(y[8 * e + 2 * k + 1]) * inv);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         stage_at(lane, c / 8 + e)),
                                     "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                     : "memory");
                    }
                } else if (row < rows) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<uint4 *>(part + part_at<ROWS>(prow, col + 4 * e)) =
                            make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            if (whole) {
                __syncwarp();
#pragma unroll
                for (int u = 0; u < CPR; ++u) {
                    const int r = (u * 32 + lane) / CPR, c = (u * 32 + lane) % CPR;
                    const int i = row - lane + r, tok = div_group(a, i);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(stage_at(r, c))
                                 : "memory");
                    const long long at =
                        (long long)(g.req.row0 + tok) * a.Hq + g.h * a.G + (i - tok * a.G);
                    if (i < rows)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * HD +
                                                   rd * NC + c * 8) = v;
                }
                __syncwarp();
            }
        }
        fence_before();
        fence_async();
        arrive_warp(bar(s.b.staged));
        if (row < rows) {
            if (!whole) {
                part[ROWS * HD + prow] = m;
                part[ROWS * HD + ROWS + prow] = l;
            } else if (a.lse) {
                const int tok = div_group(a, row);
                a.lse[(long long)(g.req.row0 + tok) * a.Hq + g.h * a.G + (row - tok * a.G)] =
                    (m + log2f(l)) * 0.69314718055994531f;
            }
        }
        if (a.count && !whole) {
            // The unit's partials are joined, kGroup at a time and in the order of the workers, by
            // the warpgroup that writes a group's last one, while the next segment streams in;
            // a group's sum takes the place of its first partial and is one of the next level's.
            // Few partials, as most units have, are one group.  A unit of a long request among
            // short ones lies in half of the workers: its groups are joined side by side.
            // the unit's first tile on the line: a worker's range begins or ends in it
            const long long begin = g.i0 > 0 ? plan.x - g.i0 : plan.x1 - g.i1;
            const int first = worker_of(begin, plan.N, plan.P);
            const int parts = worker_of(begin + sp.n - 1, plan.N, plan.P) - first + 1;
            int *count = a.count + w;
            for (int step = 1; step < parts; step *= kGroup, count += kAttnWorkers) {
                const int lo = (int)(blockIdx.x - first) / (step * kGroup) * (step * kGroup);
                const int members = min(kGroup, (parts - lo + step - 1) / step);
                if (members == 1) continue;  // its sum lies there already
                __threadfence();
                arrive_warp(bar(s.b.joined[w]));
                if (!wait(bar(s.b.joined[w]), 0, &s.dead)) return;
                if (t == 0) {
                    // No other unit's group of several begins in this worker.
                    int *here = count + (first + lo) * NWG;
                    __threadfence();
                    s.join[w] = atomicAdd(here, 1) == members - 1;
                    if (s.join[w]) *here = 0;  // for the next call
                }
                arrive_warp(bar(s.b.joined[w]));
                if (!wait(bar(s.b.joined[w]), 1, &s.dead)) return;
                if (!s.join[w]) break;  // whoever writes the group's last one goes on
                if (row >= rows) continue;
                __threadfence();
                auto slot = [&](int i) {
                    const int k = first + lo + i * step;
                    return a.part + (long long)(k == first ? 2 * k + 1 : 2 * k) * ROWS * (HD + 2);
                };
                float top = -INFINITY, total = 0.f;
                for (int i = 0; i < members; ++i) top = fmaxf(top, __ldcg(slot(i) + ROWS * HD + prow));
                const float base = top == -INFINITY ? 0.f : top;
                const bool all = step * kGroup >= parts;  // the unit's output, else a group's sum
                const int tok = div_group(a, row);
                const long long at = (long long)(g.req.row0 + tok) * a.Hq + g.h * a.G + (row - tok * a.G);
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) {
                    float o[32] = {};
                    float sum = 0.f;
#pragma unroll 2
                    for (int i = 0; i < members; ++i) {
                        const float *p = slot(i);
                        const float f = exp2f(__ldcg(p + ROWS * HD + prow) - base);
                        sum = fmaf(__ldcg(p + ROWS * HD + ROWS + prow), f, sum);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(
                                p + part_at<ROWS>(prow, c + 4 * e)));
                            o[4 * e] = fmaf(y.x, f, o[4 * e]);
                            o[4 * e + 1] = fmaf(y.y, f, o[4 * e + 1]);
                            o[4 * e + 2] = fmaf(y.z, f, o[4 * e + 2]);
                            o[4 * e + 3] = fmaf(y.w, f, o[4 * e + 3]);
                        }
                    }
                    total = sum;
                    if (all) {
                        const float inv = 1.f / sum;
                        uint4 *dst =
                            reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.o) + at * HD + c);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv),
                                                pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                                pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                                                pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
                    } else {
                        float *dst = slot(0);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            put(dst + part_at<ROWS>(prow, c + 4 * e),
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                    }
                }
                if (!all) {
                    slot(0)[ROWS * HD + prow] = top;
                    slot(0)[ROWS * HD + ROWS + prow] = total;
                } else if (a.lse) {
                    a.lse[at] = (top + log2f(total)) * 0.69314718055994531f;
                }
            }
        }
        base_slot = (base_slot + 2 * n) % C::NS;
        ++seg;
        // The last segment ends where the worker's range does.
        if (!a.count && !ahead && tid == 0)
            write_desc(a, blockIdx.x, g, !s.dead, plan.x1, plan.N, plan.P);
        arrive_warp(bar(s.b.seg_empty[seg_slot]));
    }
}

template <int HD, int NWG>
__global__ void __launch_bounds__(Cfg<HD, NWG>::kThreads, Cfg<HD, NWG>::kBlocks)
    attn_tc_kernel(const __grid_constant__ Launch L) {
    using C = Cfg<HD, NWG>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char raw[];  // the tiles first: whole swizzle atoms
    Shared &s = *reinterpret_cast<Shared *>(raw + C::kTiles);
    const uint32_t base = smem_addr(raw);
    const uint32_t qbuf = base, ring = base + NWG * C::kQTile;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(bar(s.b.full[i]), 1);
            mbar_init(bar(s.b.empty[i]), 2);  // its products, and the clearing warp
        }
        for (int w = 0; w < NWG; ++w) {
            mbar_init(bar(s.b.s_full[w]), 1);
            mbar_init(bar(s.b.p_ready[w]), 4);
            mbar_init(bar(s.b.joined[w]), 4);
            mbar_init(bar(s.b.q_ready[w]), L.q_tma ? 1 : 4);
        }
        mbar_init(bar(s.b.q_free), 1);
        for (int i = 0; i < kCleans; ++i) mbar_init(bar(s.b.clean[i]), 1);
        mbar_init(bar(s.b.o_full), 1);
        mbar_init(bar(s.b.staged), 4 * NWG);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(bar(s.b.seg_full[i]), 1);
            mbar_init(bar(s.b.seg_empty[i]), 4 * NWG + 3);  // all but the segment warp
        }
        mbar_init(bar(s.b.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s.dead = 0;
        for (int i = 0; i < 4; ++i) s.poison[i] = -1;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&L.k)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&L.v)) : "memory");
    }
    constexpr int kFirst = 4 * NWG;  // the TMA warp, then the others
    if (warp == kFirst + 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                         smem_addr(&s.tmem)),
                     "n"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Cursor cur = make_plan<C::kThreads, C::ROWS, C::KT, C::EXTRA, C::kMin>(
        L.a, blockIdx.x, gridDim.x, box_rows(L.a, C::KT), &s.plan, blockIdx.x == 0);
    __syncthreads();  // the barriers and the tensor memory's address
    fence_after();
    const uint32_t tm = *(volatile uint32_t *)&s.tmem;

    if (warp < kFirst) {
        softmax_role<HD, NWG>(L, s, qbuf, ring, tm, cur);
    } else if (warp == kFirst) {
        uint32_t issued = 0, queries = 0;
        load_role<HD, NWG>(L, s, qbuf, ring, tid & 31, issued, queries);
        // Every copy has landed before the block ends (the roles waited for them
        // unless one gave up).
        for (uint32_t p = issued > C::NS ? issued - C::NS : 0; p < issued; ++p)
            wait_parity(bar(s.b.full[p % C::NS]), (p / C::NS) & 1);
        for (int w = 0; s.dead && queries > 0 && w < NWG; ++w)
            wait_parity(bar(s.b.q_ready[w]), (queries - 1) & 1);
    } else if (warp == kFirst + 1) {
        mma_role<HD, NWG>(s, qbuf, ring, tm);
        commit(elect(), bar(s.b.drain));
        wait_parity(bar(s.b.drain), 0);
    } else if (warp == kFirst + 2) {
        if ((tid & 31) == 0) segment_role<C>(L.a, s, cur);
    } else {
        clear_role<HD, NWG>(L, s, ring, tid & 31);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (tid == 0 && s.dead && L.a.dev_err) atomicOr(L.a.dev_err, GDN_DEVERR_TIMEOUT);
    if (warp == kFirst + 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tm), "n"(C::kCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------- host side

// Pages [n_pages][kv_heads][page][hd]; boxes of 64 columns by up to a tile's places of
// one head of one page.  Pages past the end read as zeros.
bool encode_pages(CUtensorMap *map, const AttnArgs &a, const void *base, int kt) {
    const cuuint64_t page = 1ull << a.page_shift;
    const cuuint64_t dims[4] = {(cuuint64_t)a.hd, page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)a.hd * 2, page * a.hd * 2,
                                   (cuuint64_t)a.page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows(a, kt), 1, 1};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims,
                     strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [n_tok][kv_heads][group][hd], rows q_stride apart; boxes of 64 columns by 128 rows
// (token, head of one group).
bool encode_queries(CUtensorMap *map, const AttnArgs &a) {
    const cuuint64_t dims[4] = {(cuuint64_t)a.hd, (cuuint64_t)a.G, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_tok};
    const cuuint64_t strides[3] = {(cuuint64_t)a.hd * 2, (cuuint64_t)a.G * a.hd * 2,
                                   (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.G, 1, (cuuint32_t)(128 / a.G)};
    const cuuint32_t elem[4] = {1, 1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(a.q), dims, strides,
                     box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int HD, int NWG>
cudaError_t launch_tc(const AttnArgs &a, cudaStream_t stream) {
    using C = Cfg<HD, NWG>;
    Launch L;
    L.a = a;
    if (!encoder() || !encode_pages(&L.k, a, a.k, C::KT) || !encode_pages(&L.v, a, a.v, C::KT))
        return cudaErrorInvalidValue;
    L.q_tma = (a.G & (a.G - 1)) == 0 && a.G <= 128;
    if (L.q_tma && !encode_queries(&L.q, a)) return cudaErrorInvalidValue;
    constexpr int smem = C::kTiles + (int)sizeof(Shared);
    static_assert(C::kBlocks * (smem + 1024) <= 233472, "228 KB of shared memory an SM");
    const cudaError_t e = allow_smem<attn_tc_kernel<HD, NWG>>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(NWG == 2 ? kAttnTcWorkers : kAttnWorkers);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tc_kernel<HD, NWG>, L);
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, bool wide, cudaStream_t stream) {
    if (a.hd == 64) return wide ? launch_tc<64, 2>(a, stream) : launch_tc<64, 1>(a, stream);
    return wide ? launch_tc<128, 2>(a, stream) : launch_tc<128, 1>(a, stream);
}

}  // namespace gdn
