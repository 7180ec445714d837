// Linear attention with a decay for each head on the tensor cores (tcgen05): prompts (bf16, dk 64
// or 128, dv a multiple of 64).
//
// Blocks of C = 128 rows of one unit: request, head and 64 value columns.  With S the state before a
// block, G_i the sum of its first logarithms up to row i, and d(i, j) = e^{G_i - G_j}:
//     O1 = P V,   P_ij = d(i, j) (q_i . k_j) for j <= i    O2 = Q S
//     o_i = scale (O1_i + e^{G_i} O2_i)
//     U  = K^T W,  W_j = d(C - 1, j) v_j                     S <- e^{G_(C-1)} S + U
// Only S goes from block to block: everything else runs ahead of it, in roles that
// hand on through barriers:
//   TMA warp     Q, K and V tiles, ahead of their use (128-byte swizzle)
//   MMA warps    U; the other three products
//   decays       (a warp, four rows a lane) see below
//   weights      (warpgroup, a thread a row) W in two bf16 terms: each product v_j d enters its state
//                to 2^-17 of itself (a state is off by 2.3e-6; a third term, for float32's 1.2e-7, took 180 us
//                for the 133 below)
//   mask         (a thread a row) scores times decays to P, in tensor memory over the scores
//   state        (a thread a row of dk) S in registers, its bf16 copy in shared memory for O2
//   output       (a thread a row) o, which leaves by TMA
//
// Decays.  With b the 32 rows that row i is one of, and B_b the sum up to its start,
//     d(i, j) = e^{G_i - B_b} e^{B_b - G_j}:
// the first factor is left to o, so a score needs one product, with a column's factor that all of
// the 32 rows share.  For an earlier 32's rows neither exponent is positive; for its own the second
// one is, up to e^60: where the logarithms of 32 rows add up to more, their decays are products
// of single ones, taken one by one.  All sums run from their own first row; what the two exponents have in
// common cancels in the product but for its rounding, 2^-24 of up to 60: far below bf16 weights'.
// Factors of several 32s are products.  With positive logarithms these may leave float32 where the decay
// itself does not.  A block that has some is as any other while all sums within its 32s are at most 4 (what
// products of up to four then lose to underflow is below e^(16 - 87)) or within 20 of 0; else it takes each
// decay as the exponential of its own sum, out of line (709 us where it is 132; with the exponentials
// of the decays' warp alone taken so in every block it was 181).
//
// Bound by latencies from block to block, not by memory or products: 8001 rows of 32 heads take 133 us
// (64 blocks, an SM each; 39 us would be the bytes, and the tensor pipe is busy half the time there), six
// prompts of up to 4000 rows 115 us (46% of the copy's rate).  What the load pipe carries matters most,
// since barriers, products' issue and tensor memory go through it too: rows come and go by TMA
// only (queries loaded by the threads, 32 rows an instruction, 184 and 152 us against 146 and 130).  64 value
// columns a block: with 128, 8001 rows would have 32 blocks.
#include <cstdint>

#include "gdn_launch.h"
#include "gdn_linear.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int C = 128;               // rows of a block
constexpr int NV = 64;               // value columns
constexpr int kBox = C * 128;        // bytes of 64 columns of a tile
constexpr int kKeyTile = 2 * kBox;   // of queries, keys (dk = 64: the second half is not used)
constexpr int kAhead = 2;            // blocks that come to L2 before
constexpr int kThreads = 20 * 32;    // weights, mask, state, output; TMA, MMA, decays, U
constexpr float kSteep = 60.f, kRise = 4.f, kGentle = 20.f;
constexpr int kRising = 16;          // decays by their sums
constexpr int kSorted = 512;         // requests that are taken longest first
constexpr int kWTile = 2 * kBox;     // of weighted values, two terms
constexpr int kOut = 32 * 64;        // a warp's output on its way: 32 columns
constexpr int kTiles = 4 * kKeyTile + 2 * kBox + kWTile + kBox + 4 * kOut;  // Q, K, V twice; W, S

// Columns of tensor memory.
constexpr uint32_t kScores = 0, kO1 = 256, kO2 = 320, kU = 384;  // (two blocks' scores; U: two terms)

struct Bars {
    unsigned long long q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
    unsigned long long dec_full[2], dec_empty[2], s_full[2], p_ready[2];
    unsigned long long w_ready, w_free, u_full, u_free, st_ready, st_free, o_full, o_free, drain;
};

struct Shared {
    Bars b;
    struct Decays {
        alignas(16) float column[4][C];  // of an earlier or the same 32: e^{B_b - G_j} (rising: B_b - G_j)
        alignas(16) float log[C], row[C];   // (where steep) g_i, e^{G_i - B_b} (rising: G_i - B_b)
        alignas(16) float o1[C], o2[C];     // factors of O1 and O2: scale e^{G_i - B_b} (or scale), scale e^{G_i}
        alignas(16) float weight[C];        // e^{G_(C-1) - G_j}; 0 for rows past the end
        float keep;                         // e^{G_(C-1)}
        int steep;                          // a bit a 32, and kRising
    } dec[2];
    int request;
    uint32_t tmem;
    int dead;  // a wait gave up: every role leaves
};
static_assert(kTiles + sizeof(Shared) <= 232448, "227 KB of shared memory");

struct Launch {
    LinearArgs a;
    CUtensorMap q, k, v, o;
    int slices;
    bool sorted;     // ragged requests, longest first
    bool o32;        // rows are aligned to 32 bytes
    long long units;
};

// The unit of a block (one each).
struct Unit {
    int r, h, c0;  // request, head, first value column
    LinearUnit u;
    int n;         // blocks of rows
};
__device__ __forceinline__ bool find_unit(const Launch &L, const Shared &s, bool commit, Unit &x) {
    const int slice = blockIdx.x % L.slices;
    x.r = s.request;
    x.h = blockIdx.x / L.slices % L.a.g.heads;
    x.c0 = slice * NV;
    if (!linear_unit(L.a, x.r, x.h, commit, x.u)) return false;
    x.n = (x.u.T + C - 1) / C;
    return true;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(b)
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n"
                 "cp.async.bulk.commit_group;\n" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
// Into L2 only.
__device__ __forceinline__ void tma_prefetch(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}
// 32 bytes to global memory: at once where they are aligned so (rows are to 16).
__device__ __forceinline__ void stg32(void *at, bool whole, const uint32_t *x) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(x[0]),
                     "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(at)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        static_cast<uint4 *>(at)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t *x) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t *x) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3])
                 : "memory");
}
// 16 bytes c of row r of a tile's 64 columns.
__device__ __forceinline__ uint32_t chunk(uint32_t tile, int r, int c) {
    return tile + r * 128 + ((c ^ (r & 7)) << 4);
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];\n"
        : GDN_R4(r, 0), GDN_R4(r, 4), GDN_R4(r, 8), GDN_R4(r, 12)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16};\n" ::"r"(addr),
        GDN_W4(r, 0), GDN_W4(r, 4), GDN_W4(r, 8), GDN_W4(r, 12)
        : "memory");
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// The waits' slow path out of line: twenty warps in eight roles share the instruction cache.
__device__ __noinline__ bool wait_long(uint32_t b, uint32_t parity, int *dead) {
    return wait_one(b, parity, dead);
}
__device__ __forceinline__ bool await(uint32_t b, uint32_t parity, int *dead) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    return __all_sync(0xffffffffu, wait_long(b, parity, dead));
}

// Shared-memory tiles.
struct Tiles {
    uint32_t k, v, w, s, q, o;
    __device__ __forceinline__ explicit Tiles(uint32_t base)
        : k(base), v(base + 2 * kKeyTile), w(v + 2 * kBox), s(w + kWTile), q(s + kBox), o(q + 2 * kKeyTile) {}
};

// ---------------------------------------------------------------- the TMA warp (one thread)

template <bool OUT>
__device__ __forceinline__ void load_role(const Launch &L, Shared &s, const Tiles &t, uint32_t &issued) {
    const gdn_linear &g = L.a.g;
    const int boxes = g.dk / 64;
    Unit x;
    if (!find_unit(L, s, !OUT, x)) return;
    const int kx = x.h / L.a.group * g.dk, vx = x.h * g.dv + x.c0;
    for (int c = 0; c < x.n; ++c, ++issued) {
        const uint32_t slot = issued & 1, free = ((issued >> 1) & 1) ^ 1;
        const int y = x.u.row0 + c * C;
        // L2 first, some blocks before: the ring holds two, and memory takes longer than one.
        for (int a = c == 0 ? 1 : kAhead; a <= kAhead && c + a < x.n; ++a) {
            tma_prefetch(&L.v, vx, y + a * C);
            for (int b = 0; b < boxes; ++b) {
                tma_prefetch(&L.k, kx + 64 * b, y + a * C);
                if (OUT) tma_prefetch(&L.q, kx + 64 * b, y + a * C);
            }
        }
        if (OUT) {
            if (!wait_one(bar(s.b.q_empty[slot]), free, &s.dead)) return;
            arrive_expect(bar(s.b.q_full[slot]), boxes * kBox);
            for (int b = 0; b < boxes; ++b)
                tma_load(t.q + slot * kKeyTile + b * kBox, &L.q, kx + 64 * b, y, bar(s.b.q_full[slot]));
        }
        if (!wait_one(bar(s.b.k_empty[slot]), free, &s.dead)) return;
        arrive_expect(bar(s.b.k_full[slot]), boxes * kBox);
        for (int b = 0; b < boxes; ++b)
            tma_load(t.k + slot * kKeyTile + b * kBox, &L.k, kx + 64 * b, y, bar(s.b.k_full[slot]));
        if (!wait_one(bar(s.b.v_empty[slot]), free, &s.dead)) return;
        arrive_expect(bar(s.b.v_full[slot]), kBox);
        tma_load(t.v + slot * kBox, &L.v, vx, y, bar(s.b.v_full[slot]));
    }
}

// ---------------------------------------------------------------- the MMA warps

// Scores, Q S and P V.  The scores run a block ahead, so that the mask's way from scores to P is on no
// chain from block to block; U, which waits on other roles, is issued by a warp of its own.
template <int DK>
__device__ __forceinline__ void mma_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm) {
    const uint32_t lead = elect(), q_lo = desc_lo(t.q, 16), k_lo = desc_lo(t.k, 16), v_lo = desc_lo(t.v, kBox),
                   s_lo = desc_lo(t.s, kBox);
    Unit x;
    if (!find_unit(L, s, false, x)) return;
    const int n = __shfl_sync(0xffffffffu, x.n, 0);
    for (int c = -1; c < n; ++c) {
        if (c + 1 < n) {  // (P of block c - 1 was there: its product was issued before)
            const uint32_t slot = (c + 1) & 1, half = ((c + 1) >> 1) & 1;
            if (!await(bar(s.b.q_full[slot]), half, &s.dead)) return;
            if (!await(bar(s.b.k_full[slot]), half, &s.dead)) return;
            fence_after();
            const uint32_t at = slot * (kKeyTile >> 4), to = tm + kScores + slot * C;
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint32_t step = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
                mma_ss(lead, to, q_lo + at + step, k_lo + at + step, idesc(C, false), kk > 0);
            }
            commit(lead, bar(s.b.s_full[slot]));
            commit(lead, bar(s.b.k_empty[slot]));
        }
        if (c < 0) continue;
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        // O2 = Q S
        if (!await(bar(s.b.st_ready), c & 1, &s.dead)) return;
        if (!await(bar(s.b.o_free), (c & 1) ^ 1, &s.dead)) return;
        fence_after();
        const uint32_t q = q_lo + slot * (kKeyTile >> 4);
#pragma unroll
        for (int kk = 0; kk < DK / 16; ++kk)
            mma_ss(lead, tm + kO2, q + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4), s_lo + ((kk * 2048) >> 4),
                   idesc(NV, true), kk > 0);
        commit(lead, bar(s.b.st_free));
        commit(lead, bar(s.b.q_empty[slot]));
        // O1 = P V
        if (!await(bar(s.b.p_ready[slot]), half, &s.dead)) return;
        if (!await(bar(s.b.v_full[slot]), half, &s.dead)) return;
        // (values past the end are 0 by now)
        if (c + 1 == n && !await(bar(s.b.w_ready), c & 1, &s.dead)) return;
        fence_after();
        const uint32_t v = v_lo + slot * (kBox >> 4);
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
            mma_ts(lead, tm + kO1, tm + kScores + slot * C + kk * 8, v + ((kk * 2048) >> 4), idesc(NV, true), kk > 0);
        commit(lead, bar(s.b.o_full));
        commit(lead, bar(s.b.v_empty[slot]));
    }
}

// U = K^T W, both terms side by side.
template <bool OUT>
__device__ __forceinline__ void update_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm) {
    const uint32_t lead = elect(), kt_lo = desc_lo(t.k, kBox), w_lo = desc_lo(t.w, kBox);
    Unit x;
    if (!find_unit(L, s, !OUT, x)) return;
    const int n = __shfl_sync(0xffffffffu, x.n, 0);
    for (int c = 0; c < n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        if (!await(bar(s.b.k_full[slot]), half, &s.dead)) return;
        if (!await(bar(s.b.w_ready), c & 1, &s.dead)) return;
        if (!await(bar(s.b.u_free), (c & 1) ^ 1, &s.dead)) return;
        fence_after();
        const uint32_t k = kt_lo + slot * (kKeyTile >> 4);
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
            mma_ss(lead, tm + kU, k + ((kk * 2048) >> 4), w_lo + ((kk * 2048) >> 4), idesc(2 * NV, true, true),
                   kk > 0);
        commit(lead, bar(s.b.u_full));
        commit(lead, bar(s.b.w_free));
        commit(lead, bar(s.b.k_empty[slot]));
    }
}

// ---------------------------------------------------------------- the decays' warp

// Whether a block with positive logarithms needs its decays by their sums.
__device__ __forceinline__ bool rises_far(float4 x, float4 y) {
    const float high = fmaxf(fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), fmaxf(fmaxf(y.x, y.y), fmaxf(y.z, y.w)));
    const float low = fminf(fminf(fminf(x.x, x.y), fminf(x.z, x.w)), fminf(fminf(y.x, y.y), fminf(y.z, y.w)));
    const bool number = !isnan(x.x + x.y + x.z + x.w + y.x + y.y + y.z + y.w);
    return !__all_sync(0xffffffffu, number && high <= kRise) &&
           !__all_sync(0xffffffffu, number && high <= kGentle && low >= -kGentle);
}

// A block's decays where its logarithms rise: sums, or exponentials of whole sums.  This lane's rows as below.
template <bool OUT>
__device__ __noinline__ bool rising_decays(Shared::Decays &d, float scale, int lane, int n, float4 gl, float4 upto,
                                           float4 after, float total) {
    if (!rises_far(upto, after)) return false;
    const int b = lane >> 3, i = 4 * lane;
    float before = 0.f, behind = 0.f, all = 0.f;
    auto put = [&](float *to, float w, float x, float y, float z) {
        *reinterpret_cast<float4 *>(to + i) = make_float4(w, x, y, z);
    };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float sum = __shfl_sync(0xffffffffu, total, 8 * m);
        all += sum;
        if (m < b) before += sum;
        if (m > b) {
            if (OUT)
                put(d.column[m], after.x + behind, after.y + behind, after.z + behind, after.w + behind);
            behind += sum;
        }
    }
    put(d.weight, i < n ? expf(after.x + behind) : 0.f, i + 1 < n ? expf(after.y + behind) : 0.f,
        i + 2 < n ? expf(after.z + behind) : 0.f, i + 3 < n ? expf(after.w + behind) : 0.f);
    if (OUT) {
        put(d.log, gl.x, gl.y, gl.z, gl.w);
        put(d.row, upto.x, upto.y, upto.z, upto.w);
        put(d.o1, scale, scale, scale, scale);
        put(d.o2, scale * expf(before + upto.x), scale * expf(before + upto.y), scale * expf(before + upto.z),
            scale * expf(before + upto.w));
    }
    if (lane == 0) {
        d.keep = expf(all);
        d.steep = kRising;
    }
    return true;
}

template <bool OUT>
__device__ __forceinline__ void decay_role(const Launch &L, Shared &s, int lane) {
    const gdn_linear &g = L.a.g;
    const int b = lane >> 3, l = lane & 7;  // this lane's rows: 4 lane to 4 lane + 3, of the 32 that are b
    Unit x;
    float next[4];
    if (!find_unit(L, s, !OUT, x)) return;
    auto load = [&](int c) {  // 0 for rows past the end
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int row = c * C + 4 * lane + k;
            next[k] = row < x.u.T ? __ldg(g.log_decay + (x.u.row0 + (long long)row) * g.decay_stride + x.h) : 0.f;
        }
    };
    load(0);
    for (int c = 0; c < x.n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        const int n = min(C, x.u.T - c * C);
        const float gl[4] = {next[0], next[1], next[2], next[3]};
        if (c + 1 < x.n) load(c + 1);
        // Sums within the 32: from its start up to each row, and from behind it to the end.
        float upto[4] = {gl[0], gl[0] + gl[1], 0.f, 0.f}, after[4] = {0.f, 0.f, gl[3], 0.f};
        upto[2] = upto[1] + gl[2];
        upto[3] = upto[2] + gl[3];
        after[1] = after[2] + gl[2];
        after[0] = after[1] + gl[1];
        float below = upto[3], above = upto[3];
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, below, d, 8);
            const float z = __shfl_down_sync(0xffffffffu, above, d, 8);
            if (l >= d) below += y;
            if (l + d < 8) above += z;
        }
        const float total = __shfl_sync(0xffffffffu, below, lane | 7);
        below = __shfl_up_sync(0xffffffffu, below, 1, 8);
        above = __shfl_down_sync(0xffffffffu, above, 1, 8);
        if (l == 0) below = 0.f;
        if (l == 7) above = 0.f;
        bool mild = true;
        const bool falls =  // (false for NaN)
            gl[0] <= 0.f && gl[1] <= 0.f && gl[2] <= 0.f && gl[3] <= 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            upto[k] += below;
            after[k] += above;
            mild = mild && fabsf(upto[k]) < kSteep;  // (false for NaN)
        }
        const unsigned steep = ~__ballot_sync(0xffffffffu, mild);
        const bool steep_here = (steep >> (8 * b) & 0xFFu) != 0;
        const float whole = expf(total);
        float t[4];  // of the four 32s
#pragma unroll
        for (int m = 0; m < 4; ++m) t[m] = __shfl_sync(0xffffffffu, whole, 8 * m);
        float row[4], col[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            row[k] = expf(upto[k]);
            col[k] = expf(after[k]);
        }
        const bool falls_all = __all_sync(0xffffffffu, falls);
        if (!await(bar(s.b.dec_empty[slot]), half ^ 1, &s.dead)) return;
        Shared::Decays &d = s.dec[slot];
        if (!falls_all && rising_decays<OUT>(d, g.scale, lane, n, make_float4(gl[0], gl[1], gl[2], gl[3]),
                                             make_float4(upto[0], upto[1], upto[2], upto[3]),
                                             make_float4(after[0], after[1], after[2], after[3]), total)) {
            arrive_warp(bar(s.b.dec_full[slot]));
            continue;
        }
        auto put = [&](float *to, float w, float x, float y, float z) {
            *reinterpret_cast<float4 *>(to + 4 * lane) = make_float4(w, x, y, z);
        };
        float f = 1.f;
#pragma unroll
        for (int m = 1; m < 4; ++m) {
            if (m <= b) continue;  // the rows of earlier 32s do not see this one
            if (OUT) put(d.column[m], f * col[0], f * col[1], f * col[2], f * col[3]);
            f *= t[m];
        }
        const int i = 4 * lane;
        put(d.weight, i < n ? f * col[0] : 0.f, i + 1 < n ? f * col[1] : 0.f, i + 2 < n ? f * col[2] : 0.f,
            i + 3 < n ? f * col[3] : 0.f);
        if (OUT) {
            put(d.column[b], expf(-upto[0]), expf(-upto[1]), expf(-upto[2]), expf(-upto[3]));
            float e = g.scale;
#pragma unroll
            for (int m = 0; m < 3; ++m)
                if (m < b) e *= t[m];
            put(d.o2, e * row[0], e * row[1], e * row[2], e * row[3]);
            if (steep_here) {
                put(d.log, gl[0], gl[1], gl[2], gl[3]);
                put(d.row, row[0], row[1], row[2], row[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) row[k] = 1.f;
            }
            put(d.o1, g.scale * row[0], g.scale * row[1], g.scale * row[2], g.scale * row[3]);
        }
        if (lane == 0) {
            d.keep = t[0] * t[1] * (t[2] * t[3]);
            d.steep = ((steep & 0xFFu) != 0) | ((steep >> 8 & 0xFFu) != 0) << 1 |
                      ((steep >> 16 & 0xFFu) != 0) << 2 | ((steep >> 24) != 0) << 3;
        }
        arrive_warp(bar(s.b.dec_full[slot]));
    }
}

// ---------------------------------------------------------------- the weights' warpgroup

template <bool OUT>
__device__ __forceinline__ void weight_role(const Launch &L, Shared &s, const Tiles &t, int j) {
    const gdn_linear &g = L.a.g;
    Unit x;
    if (!find_unit(L, s, !OUT, x)) return;
    for (int c = 0; c < x.n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        const int n = min(C, x.u.T - c * C);
        if (!await(bar(s.b.dec_full[slot]), half, &s.dead)) return;
        const float w = s.dec[slot].weight[j];
        arrive_warp(bar(s.b.dec_empty[slot]));
        if (!await(bar(s.b.v_full[slot]), half, &s.dead)) return;
        const uint32_t vt = t.v + slot * kBox;
        const uint32_t zero[4] = {0, 0, 0, 0};
        if (n < C) {  // rows of other requests, whatever they hold, count as 0
            if (!await(bar(s.b.k_full[slot]), half, &s.dead)) return;
            if (j >= n) {
                for (int e = 0; e < 8; ++e) {
                    sts128(chunk(vt, j, e), zero);
                    for (int box = 0; box < g.dk / 64; ++box)
                        sts128(chunk(t.k + slot * kKeyTile + box * kBox, j, e), zero);
                }
            }
        }
        const float2 w2 = make_float2(w, w);
        uint32_t v8[8][4];
#pragma unroll
        for (int e = 0; e < 8; ++e) lds128(chunk(vt, j, e), v8[e]);
        arrive_warp(bar(s.b.v_empty[slot]));
        if (!await(bar(s.b.w_free), (c & 1) ^ 1, &s.dead)) return;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t *v = v8[e], hi[4], lo[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 y = mul2(make_float2(__uint_as_float(v[m] << 16),
                                                  __uint_as_float(v[m] & 0xFFFF0000u)), w2);
                hi[m] = pack_bf16(y.x, y.y);
                const float2 z = add2(y, make_float2(-__uint_as_float(hi[m] << 16),
                                                     -__uint_as_float(hi[m] & 0xFFFF0000u)));
                lo[m] = pack_bf16(z.x, z.y);
            }
            sts128(chunk(t.w, j, e), hi);
            sts128(chunk(t.w + kBox, j, e), lo);
        }
        fence_async();
        arrive_warp(bar(s.b.w_ready));
    }
}

// ---------------------------------------------------------------- the mask's warpgroup

// A warp's rows in a block whose logarithms rise: each decay the exponential of its sum.
__device__ __noinline__ void mask_rising(const Shared::Decays &d, uint32_t ts, int lane, int b) {
    const float f = d.row[32 * b + lane];
#pragma unroll 1
    for (int m = 0; m <= b; ++m) {
        uint32_t y[32];
        tmem_ld32(ts + 32 * m, y);
        wait_ld();
        float sum = 0.f;
#pragma unroll
        for (int e = 31; e >= 0; --e) {
            if (m < b)
                sum = d.column[b][32 * m + e] + f;
            else if (e < lane)
                sum += d.log[32 * b + e + 1];
            y[e] = m < b || e <= lane ? __float_as_uint(__uint_as_float(y[e]) * expf(sum)) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            y[e / 2] = pack_bf16(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
        tmem_st16(ts + 16 * m, y);  // over scores that have been read
    }
}

// A warp's rows whose 32 is steep: the factors of earlier 32s' columns times the row's, and its own
// decays one by one.  (A function of its own, so that its registers are not the others'.)
__device__ __noinline__ void mask_steep(const Shared::Decays &d, uint32_t ts, int lane, int b) {
    const float f = d.row[32 * b + lane];
#pragma unroll 1
    for (int m = 0; m <= b; ++m) {
        uint32_t y[32];
        tmem_ld32(ts + 32 * m, y);
        wait_ld();
        if (m < b) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                y[e] = __float_as_uint(__uint_as_float(y[e]) * (d.column[b][32 * m + e] * f));
        } else {
            float p = 1.f;
#pragma unroll
            for (int e = 31; e >= 0; --e) {
                if (e < lane) p *= expf(d.log[32 * b + e + 1]);
                y[e] = e <= lane ? __float_as_uint(__uint_as_float(y[e]) * p) : 0u;
            }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2)
            y[e / 2] = pack_bf16(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
        tmem_st16(ts + 16 * m, y);  // over scores that have been read
    }
}

__device__ __forceinline__ void mask_role(const Launch &L, Shared &s, uint32_t tm, int i) {
    const int lane = i & 31, b = i >> 5;
    Unit x;
    if (!find_unit(L, s, false, x)) return;
    for (int c = 0; c < x.n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        if (!await(bar(s.b.dec_full[slot]), half, &s.dead)) return;
        const Shared::Decays &d = s.dec[slot];
        if (!await(bar(s.b.s_full[slot]), half, &s.dead)) return;
        const uint32_t ts = tm + kScores + slot * C + ((uint32_t)b << 21);  // this warp's lanes
        fence_after();
        if (d.steep & kRising) {
            mask_rising(d, ts, lane, b);
        } else if (d.steep >> b & 1) {
            mask_steep(d, ts, lane, b);
        } else {
#pragma unroll 1
            for (int m = 0; m <= b; ++m) {
                uint32_t y[32];
                tmem_ld32(ts + 32 * m, y);
                const float *column = d.column[b] + 32 * m;
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(column + e);
                    const float2 p0 = mul2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])),
                                           make_float2(w.x, w.y));
                    const float2 p1 = mul2(make_float2(__uint_as_float(y[e + 2]), __uint_as_float(y[e + 3])),
                                           make_float2(w.z, w.w));
                    y[e / 2] = pack_bf16(p0.x, p0.y);
                    y[e / 2 + 1] = pack_bf16(p1.x, p1.y);
                }
                if (m == b) {  // its own 32: up to itself
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] &= (2 * e <= lane ? 0xFFFFu : 0u) | (2 * e + 1 <= lane ? 0xFFFF0000u : 0u);
                }
                tmem_st16(ts + 16 * m, y);  // over scores that have been read
            }
        }
        uint32_t zero[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll 1
        for (int m = b + 1; m < 4; ++m) tmem_st16(ts + 16 * m, zero);
        arrive_warp(bar(s.b.dec_empty[slot]));
        wait_st();
        fence_before();
        arrive_warp(bar(s.b.p_ready[slot]));
    }
}

// ---------------------------------------------------------------- the state's warpgroup

template <bool OUT, bool STATE>
__device__ __forceinline__ void state_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm, int d) {
    const gdn_linear &g = L.a.g;
    const uint32_t tu = tm + kU + ((uint32_t)(d >> 5) << 21);
    Unit x;
    if (!find_unit(L, s, !OUT, x)) return;
    float *row = x.u.tile + (long long)d * g.dv + x.c0;
    float S[NV];
#pragma unroll
    for (int e = 0; e < NV; e += 4) {
        const float4 y = d < g.dk ? __ldcs(reinterpret_cast<const float4 *>(row + e))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
        S[e] = y.x;
        S[e + 1] = y.y;
        S[e + 2] = y.z;
        S[e + 3] = y.w;
    }
    for (int c = 0; c < x.n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        if (OUT) {
            if (!await(bar(s.b.st_free), (c & 1) ^ 1, &s.dead)) return;
            if (d < g.dk) {
#pragma unroll
                for (int e = 0; e < NV; e += 8) {
                    const uint32_t y[4] = {pack_bf16(S[e], S[e + 1]), pack_bf16(S[e + 2], S[e + 3]),
                                           pack_bf16(S[e + 4], S[e + 5]), pack_bf16(S[e + 6], S[e + 7])};
                    sts128(chunk(t.s, d, e / 8), y);
                }
            }
            fence_async();
            arrive_warp(bar(s.b.st_ready));
        }
        if (!await(bar(s.b.dec_full[slot]), half, &s.dead)) return;
        const float keep = s.dec[slot].keep;
        arrive_warp(bar(s.b.dec_empty[slot]));
        if (!await(bar(s.b.u_full), c & 1, &s.dead)) return;
        fence_after();
#pragma unroll
        for (int e = 0; e < NV; e += 16) {
            uint32_t y[16], z[16];
            tmem_ld16(tu + e, y);
            tmem_ld16(tu + NV + e, z);
            wait_ld();
#pragma unroll
            for (int m = 0; m < 16; m += 2) {
                const float2 u = add2(make_float2(__uint_as_float(y[m]), __uint_as_float(y[m + 1])),
                                      make_float2(__uint_as_float(z[m]), __uint_as_float(z[m + 1])));
                const float2 w = fma2(make_float2(S[e + m], S[e + m + 1]), make_float2(keep, keep), u);
                S[e + m] = w.x;
                S[e + m + 1] = w.y;
            }
        }
        fence_before();
        arrive_warp(bar(s.b.u_free));
    }
    if (STATE && d < g.dk) {
#pragma unroll
        for (int e = 0; e < NV; e += 4)
            __stcs(reinterpret_cast<float4 *>(row + e), make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]));
    }
}

// ---------------------------------------------------------------- the output's warpgroup

__device__ __forceinline__ void output_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm, int i) {
    const gdn_linear &g = L.a.g;
    const int b = i >> 5;
    const uint32_t lanes = (uint32_t)b << 21, out = t.o + b * kOut;
    Unit x;
    if (!find_unit(L, s, false, x)) return;
    for (int c = 0; c < x.n; ++c) {
        const uint32_t slot = c & 1, half = (c >> 1) & 1;
        const int n = min(C, x.u.T - c * C);
        if (!await(bar(s.b.dec_full[slot]), half, &s.dead)) return;
        const float f = s.dec[slot].o2[i], f1 = s.dec[slot].o1[i];
        arrive_warp(bar(s.b.dec_empty[slot]));
        if (!await(bar(s.b.o_full), c & 1, &s.dead)) return;
        fence_after();
        const float2 f2 = make_float2(f, f), scale2 = make_float2(f1, f1);
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(L.a.o) +
                           (x.u.row0 + (long long)c * C + i) * g.heads * g.dv + x.h * g.dv + x.c0;
#pragma unroll
        for (int h = 0; h < NV; h += 32) {
            uint32_t y[32], z[32];
            tmem_ld32(tm + kO1 + lanes + h, y);
            tmem_ld32(tm + kO2 + lanes + h, z);
            wait_ld();
            if (h + 32 == NV) {
                fence_before();
                arrive_warp(bar(s.b.o_free));
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                const float2 p = fma2(make_float2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])), f2,
                                      mul2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), scale2));
                y[e / 2] = pack_bf16(p.x, p.y);
            }
            if (n == C) {  // 32 rows and columns a warp leave by TMA
                const int lane = i & 31;
                if (lane == 0) tma_stores_read();  // the last ones have
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 4; ++e) sts128(out + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4), y + 4 * e);
                fence_async();
                __syncwarp();
                if (lane == 0) tma_store(&L.o, x.h * g.dv + x.c0 + h, x.u.row0 + c * C + i, out);
            } else if (i < n) {  // whole sectors: 32 bytes of a row at a time
                stg32(o + h, L.o32, y);
                stg32(o + h + 16, L.o32, y + 8);
            }
        }
    }
}

// ---------------------------------------------------------------- kernel

template <int MODE>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ Launch L) {
    constexpr bool OUT = MODE != kCommit, STATE = MODE != kVerify;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char raw[];  // the tiles first: whole swizzle atoms
    Shared &s = *reinterpret_cast<Shared *>(raw + kTiles);
    const Tiles t(smem_addr(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(s.b.q_full[i]), 1);
            mbar_init(bar(s.b.q_empty[i]), 1);
            mbar_init(bar(s.b.k_full[i]), 1);
            mbar_init(bar(s.b.k_empty[i]), OUT ? 2 : 1);
            mbar_init(bar(s.b.v_full[i]), 1);
            mbar_init(bar(s.b.v_empty[i]), OUT ? 5 : 4);
            mbar_init(bar(s.b.dec_full[i]), 1);
            mbar_init(bar(s.b.dec_empty[i]), OUT ? 16 : 8);
            mbar_init(bar(s.b.s_full[i]), 1);
            mbar_init(bar(s.b.p_ready[i]), 4);
        }
        mbar_init(bar(s.b.w_ready), 4);
        mbar_init(bar(s.b.w_free), 1);
        mbar_init(bar(s.b.u_full), 1);
        mbar_init(bar(s.b.u_free), 4);
        mbar_init(bar(s.b.st_ready), 4);
        mbar_init(bar(s.b.st_free), 1);
        mbar_init(bar(s.b.o_full), 1);
        mbar_init(bar(s.b.o_free), 4);
        mbar_init(bar(s.b.drain), OUT ? 2 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s.dead = 0;
    }
    if (warp == 17) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                         smem_addr(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const gdn_linear &g = L.a.g;
    const int rank = blockIdx.x / L.slices / g.heads;
    if (L.sorted) {  // (lengths where tiles will be)
        int *length = reinterpret_cast<int *>(raw);
        for (int i = tid; i < g.batch; i += kThreads) length[i] = g.cu_seqlens[i + 1] - g.cu_seqlens[i];
        __syncthreads();
        for (int i = tid; i < g.batch; i += kThreads) {
            int before = 0;
            for (int k = 0; k < g.batch; ++k) before += length[k] > length[i] || (length[k] == length[i] && k < i);
            if (before == rank) s.request = i;
        }
        fence_async();
    } else if (tid == 0) {
        s.request = rank;
    }
    __syncthreads();  // the barriers and the tensor memory's address
    fence_after();
    const uint32_t tm = *(volatile uint32_t *)&s.tmem;

    if (warp < 4) {
        weight_role<OUT>(L, s, t, tid);
    } else if (warp < 8) {
        if (OUT) mask_role(L, s, tm, tid - 128);
    } else if (warp < 12) {
        state_role<OUT, STATE>(L, s, t, tm, tid - 256);
    } else if (warp < 16) {
        if (OUT) {
            output_role(L, s, t, tm, tid - 384);
            if ((tid & 31) == 0) tma_stores_read();
        }
    } else if (warp == 18) {
        decay_role<OUT>(L, s, tid & 31);
    } else if (warp == 16) {
        if ((tid & 31) == 0) {
            uint32_t issued = 0;
            load_role<OUT>(L, s, t, issued);
            // Every copy has landed before the block ends (its roles waited for them unless one gave up; then those
            // of a block of rows that was asked for in part may be on their way too, and its other waits run out).
            for (uint32_t p = issued > 2 ? issued - 2 : 0; p < issued + (s.dead ? 1 : 0); ++p) {
                wait_parity(bar(s.b.v_full[p & 1]), (p >> 1) & 1);
                wait_parity(bar(s.b.k_full[p & 1]), (p >> 1) & 1);
                if (OUT) wait_parity(bar(s.b.q_full[p & 1]), (p >> 1) & 1);
            }
        }
    } else {
        if (warp == 19) {
            update_role<OUT>(L, s, t, tm);
        } else if (OUT) {
            if (L.a.g.dk == 128)
                mma_role<128>(L, s, t, tm);
            else
                mma_role<64>(L, s, t, tm);
        }
        if (OUT || warp == 19) commit(elect(), bar(s.b.drain));
        wait_parity(bar(s.b.drain), 0);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (tid == 0 && s.dead && L.a.g.dev_err) atomicOr(L.a.g.dev_err, GDN_DEVERR_TIMEOUT);
    if (warp == 17) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tm) : "memory");
    }
}

// ---------------------------------------------------------------- host side

// Rows of `cols` elements, `stride` apart; boxes of 64 columns (or 32).  Rows past the end read as zeros.
bool encode_rows(CUtensorMap *map, const void *base, long long cols, long long rows, long long stride,
                 unsigned box_rows = C, unsigned box_cols = 64) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t elem[2] = {1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                     elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_tc(const LinearArgs &a, cudaStream_t stream) {
    const gdn_linear &g = a.g;
    Launch L;
    L.a = a;
    L.slices = g.dv / NV;
    L.o32 = (reinterpret_cast<uintptr_t>(a.o) & 31) == 0;
    L.units = (long long)g.batch * g.heads * L.slices;
    L.sorted = g.cu_seqlens && g.batch > 1 && g.batch <= kSorted && L.units > 152;
    const long long krow = (long long)g.k_heads * g.dk, vrow = (long long)g.heads * g.dv;
    if (!encoder() || (MODE != kCommit && !encode_rows(&L.q, g.q, krow, g.n_tok, g.q_stride)) ||
        !encode_rows(&L.k, g.k, krow, g.n_tok, g.k_stride) ||
        !encode_rows(&L.v, g.v, vrow, g.n_tok, g.v_stride) ||
        (MODE != kCommit && !encode_rows(&L.o, a.o, vrow, g.n_tok, vrow, 32, 32)))
        return cudaErrorInvalidValue;
    constexpr int smem = kTiles + (int)sizeof(Shared);
    const cudaError_t e = allow_smem<linear_tc_kernel<MODE>>(smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)L.units);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_tc_kernel<MODE>, L);
}

}  // namespace

bool linear_tc_runs(const gdn_linear &g) {
    // The tensor maps' strides are below 2^40 bytes, as those that validation lets through are.
    return g.dtype == GDN_BF16 && (g.dk == 64 || g.dk == 128) && g.dv % NV == 0 && g.max_T >= kLinearTcRows;
}

cudaError_t launch_linear_tc(const LinearArgs &a, int mode, cudaStream_t stream) {
    switch (mode) {
        case kVerify: return launch_tc<kVerify>(a, stream);
        case kCommit: return launch_tc<kCommit>(a, stream);
        default: return launch_tc<kFused>(a, stream);
    }
}

}  // namespace gdn
