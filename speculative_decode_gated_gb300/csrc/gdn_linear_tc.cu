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
//   TMA warp     Q, K and V tiles, two blocks ahead (128-byte swizzle)
//   MMA warp     the four products
//   weights      (warpgroup, a thread a row) the decays, and W in three bf16 terms, which hold
//                the float32 product v_j d whole: a state is as exact as its float32 sums
//   mask         (a thread a row) scores times decays to P, in tensor memory over the scores
//   state        (a thread a row of dk) S in registers, its bf16 copy in shared memory for O2
//   output       (a thread a row) o, through the block's Q tile, and by TMA to global memory
//
// Decays.  No exponent is positive and nothing cancels: within a warp's 32 rows, e^{...} of sums
// taken from the row to the end of the 32 (cf) or from their start to the row (rowf); t, those
// of whole 32s.  d(i, j) = cf_j (t of the 32s between) rowf_i; within the 32, products of
// single decays.
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
constexpr int kThreads = 18 * 32;    // weights, mask, state, output; TMA, MMA
constexpr int kTiles = 4 * kKeyTile + 2 * kBox + 3 * kBox + kBox;  // Q, K: 2; V: 2; W: 3 terms; S

// Columns of tensor memory.
constexpr uint32_t kScores = 0, kO1 = 256, kO2 = 320, kU = 384;

struct Bars {
    unsigned long long q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
    unsigned long long dec_full[2], dec_empty[2], s_full[2], p_ready[2], u_full[2], u_free[2];
    unsigned long long w_ready, w_free, st_ready, st_free, o_full, o_free, w_sync, o_sync, drain;
};

struct Shared {
    Bars b;
    alignas(16) float cf[2][C];  // read four at a time
    float rowf[2][C], t[2][4];
    uint32_t tmem;
    int dead;  // a wait gave up: every role leaves
};
static_assert(kTiles + sizeof(Shared) <= 232448, "227 KB of shared memory");

struct Launch {
    LinearArgs a;
    CUtensorMap q, k, v, o;
    int slices;
    long long units;
};

// The units of a block, in order.
struct Unit {
    int r, h, c0;  // request, head, first value column
    LinearUnit u;
    int n;         // blocks of rows
};
__device__ __forceinline__ bool next_unit(const Launch &L, bool commit, long long &at, Unit &x) {
    for (; at < L.units; at += gridDim.x) {
        const int s = (int)(at % L.slices);
        const long long rh = at / L.slices;
        x.r = (int)(rh / L.a.g.heads);
        x.h = (int)(rh - (long long)x.r * L.a.g.heads);
        x.c0 = s * NV;
        if (linear_unit(L.a, x.r, x.h, commit, x.u)) {
            x.n = (x.u.T + C - 1) / C;
            at += gridDim.x;
            return true;
        }
    }
    return false;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(b)
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap *map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
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

// Shared-memory tiles.
struct Tiles {
    uint32_t q, k, v, w, s;
    __device__ __forceinline__ explicit Tiles(uint32_t base)
        : q(base), k(base + 2 * kKeyTile), v(base + 4 * kKeyTile), w(v + 2 * kBox), s(w + 3 * kBox) {}
};

// The logarithm of row i's decay (0 for rows past the block's end).
__device__ __forceinline__ float log_decay(const gdn_linear &g, const Unit &x, int c, int i) {
    const int row = c * C + i;
    return row < x.u.T ? __ldg(g.log_decay + (x.u.row0 + (long long)row) * g.decay_stride + x.h) : 0.f;
}

// ---------------------------------------------------------------- the TMA warp (one thread)

template <bool OUT>
__device__ __forceinline__ void load_role(const Launch &L, Shared &s, const Tiles &t, uint32_t &issued) {
    const gdn_linear &g = L.a.g;
    const int boxes = g.dk / 64;
    long long at = blockIdx.x;
    Unit x;
    while (next_unit(L, !OUT, at, x)) {
        const int kx = x.h / L.a.group * g.dk, vx = x.h * g.dv + x.c0;
        for (int c = 0; c < x.n; ++c, ++issued) {
            const uint32_t slot = issued & 1, free = ((issued >> 1) & 1) ^ 1;
            const int y = x.u.row0 + c * C;
            auto keys = [&](const CUtensorMap *map, uint32_t dst, unsigned long long &full,
                            unsigned long long &empty) {
                if (!wait_one(bar(empty), free, &s.dead)) return false;
                arrive_expect(bar(full), boxes * kBox);
                for (int b = 0; b < boxes; ++b)
                    tma_load(dst + slot * kKeyTile + b * kBox, map, kx + 64 * b, y, bar(full));
                return true;
            };
            if (!wait_one(bar(s.b.v_empty[slot]), free, &s.dead)) return;
            arrive_expect(bar(s.b.v_full[slot]), kBox);
            tma_load(t.v + slot * kBox, &L.v, vx, y, bar(s.b.v_full[slot]));
            if (!keys(&L.k, t.k, s.b.k_full[slot], s.b.k_empty[slot])) return;
            if (OUT && !keys(&L.q, t.q, s.b.q_full[slot], s.b.q_empty[slot])) return;
        }
    }
}

// ---------------------------------------------------------------- the MMA warp

template <bool OUT>
__device__ __forceinline__ void mma_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm) {
    const uint32_t lead = elect();
    const int steps = __shfl_sync(0xffffffffu, L.a.g.dk / 16, 0);
    const uint32_t q_lo = desc_lo(t.q, 16), k_lo = desc_lo(t.k, 16);  // rows of 64 columns
    const uint32_t kt_lo = desc_lo(t.k, kBox);                        // K^T, 128 of its rows
    const uint32_t v_lo = desc_lo(t.v, kBox), w_lo = desc_lo(t.w, kBox), s_lo = desc_lo(t.s, kBox);
    tm = __shfl_sync(0xffffffffu, tm, 0);
    long long at = blockIdx.x;
    Unit x;
    uint32_t it = 0;  // blocks so far
    auto scores = [&](uint32_t i) -> bool {
        const uint32_t slot = i & 1, full = (i >> 1) & 1;
        if (!wait(bar(s.b.q_full[slot]), full, &s.dead)) return false;
        if (!wait(bar(s.b.k_full[slot]), full, &s.dead)) return false;
        fence_after();
        for (int kk = 0; kk < steps; ++kk) {
            const uint32_t off = (slot * kKeyTile + (kk >> 2) * kBox + (kk & 3) * 32) >> 4;
            mma_ss(lead, tm + kScores + slot * 128, q_lo + off, k_lo + off, idesc(C, false), kk > 0);
        }
        commit(lead, bar(s.b.s_full[slot]));
        return true;
    };
    while (next_unit(L, !OUT, at, x)) {
        const int n = __shfl_sync(0xffffffffu, x.n, 0);
        if (OUT && !scores(it)) return;
        for (int c = 0; c < n; ++c, ++it) {
            const uint32_t slot = it & 1, half = (it >> 1) & 1;
            // U = K^T W
            if (!wait(bar(s.b.k_full[slot]), half, &s.dead)) return;
            if (!wait(bar(s.b.w_ready), it & 1, &s.dead)) return;
            if (!wait(bar(s.b.u_free[slot]), half ^ 1, &s.dead)) return;
            fence_after();
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk)
                    mma_ss(lead, tm + kU + slot * NV, kt_lo + ((slot * kKeyTile + kk * 2048) >> 4),
                           w_lo + ((p * kBox + kk * 2048) >> 4), idesc(NV, true, true), p + kk > 0);
            commit(lead, bar(s.b.u_full[slot]));
            commit(lead, bar(s.b.w_free));
            commit(lead, bar(s.b.k_empty[slot]));
            if (!OUT) {
                commit(lead, bar(s.b.v_empty[slot]));
                continue;
            }
            if (c + 1 < n && !scores(it + 1)) return;
            // O2 = Q S
            if (!wait(bar(s.b.st_ready), it & 1, &s.dead)) return;
            if (!wait(bar(s.b.o_free), (it & 1) ^ 1, &s.dead)) return;
            fence_after();
            for (int kk = 0; kk < steps; ++kk)
                mma_ss(lead, tm + kO2, q_lo + ((slot * kKeyTile + (kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                       s_lo + ((kk * 2048) >> 4), idesc(NV, true), kk > 0);
            commit(lead, bar(s.b.st_free));
            // O1 = P V
            if (!wait(bar(s.b.p_ready[slot]), half, &s.dead)) return;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk)
                mma_ts(lead, tm + kO1, tm + kScores + slot * 128 + kk * 8,
                       v_lo + ((slot * kBox + kk * 2048) >> 4), idesc(NV, true), kk > 0);
            commit(lead, bar(s.b.o_full));
            commit(lead, bar(s.b.v_empty[slot]));
        }
    }
}

// ---------------------------------------------------------------- the weights' warpgroup

template <bool OUT>
__device__ __forceinline__ void weight_role(const Launch &L, Shared &s, const Tiles &t, int j) {
    const gdn_linear &g = L.a.g;
    const int lane = j & 31, b = j >> 5;
    long long at = blockIdx.x;
    Unit x;
    uint32_t it = 0;
    while (next_unit(L, !OUT, at, x)) {
        float gj = log_decay(g, x, 0, j);
        for (int c = 0; c < x.n; ++c, ++it) {
            const uint32_t slot = it & 1, half = (it >> 1) & 1;
            const int n = min(C, x.u.T - c * C);
            float upto = gj, after = __shfl_down_sync(0xffffffffu, gj, 1);
            if (lane == 31) after = 0.f;
            if (c + 1 < x.n) gj = log_decay(g, x, c + 1, j);
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, upto, d);
                const float z = __shfl_down_sync(0xffffffffu, after, d);
                if (lane >= d) upto += y;
                if (lane + d < 32) after += z;
            }
            const float cf = expf(after);
            if (!wait(bar(s.b.dec_empty[slot]), half ^ 1, &s.dead)) return;
            const float rowf = expf(upto);
            s.rowf[slot][j] = rowf;
            s.cf[slot][j] = cf;
            if (lane == 31) s.t[slot][b] = rowf;
            arrive_warp(bar(s.b.dec_full[slot]));
            arrive_warp(bar(s.b.w_sync));
            if (!wait(bar(s.b.w_sync), it & 1, &s.dead)) return;
            float w = cf;
#pragma unroll
            for (int m = 1; m < 4; ++m)
                if (m > b) w *= s.t[slot][m];
            if (!wait(bar(s.b.v_full[slot]), half, &s.dead)) return;
            if (!wait(bar(s.b.w_free), (it & 1) ^ 1, &s.dead)) return;
            const uint32_t vt = t.v + slot * kBox;
            const uint32_t zero[4] = {0, 0, 0, 0};
            if (n < C) {  // rows of other requests, whatever they hold, count as 0
                if (!wait(bar(s.b.k_full[slot]), half, &s.dead)) return;
                if (j >= n) {
                    for (int e = 0; e < 8; ++e) {
                        sts128(chunk(vt, j, e), zero);
                        for (int box = 0; box < g.dk / 64; ++box)
                            sts128(chunk(t.k + slot * kKeyTile + box * kBox, j, e), zero);
                    }
                }
            }
            const float2 w2 = make_float2(w, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t v[4], hi[4], mid[4], lo[4];
                lds128(chunk(vt, j, e), v);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float2 y = mul2(make_float2(__uint_as_float(v[m] << 16),
                                                      __uint_as_float(v[m] & 0xFFFF0000u)), w2);
                    // the leading 8 bits of each, the next 8 and the last 8: exact
                    const uint32_t yx = __float_as_uint(y.x), yy = __float_as_uint(y.y);
                    hi[m] = __byte_perm(yx, yy, 0x7632);
                    const float2 y1 = add2(y, make_float2(-__uint_as_float(yx & 0xFFFF0000u),
                                                          -__uint_as_float(yy & 0xFFFF0000u)));
                    const uint32_t zx = __float_as_uint(y1.x), zy = __float_as_uint(y1.y);
                    mid[m] = __byte_perm(zx, zy, 0x7632);
                    const float2 y2 = add2(y1, make_float2(-__uint_as_float(zx & 0xFFFF0000u),
                                                           -__uint_as_float(zy & 0xFFFF0000u)));
                    lo[m] = pack_bf16(y2.x, y2.y);
                }
                sts128(chunk(t.w, j, e), hi);
                sts128(chunk(t.w + kBox, j, e), mid);
                sts128(chunk(t.w + 2 * kBox, j, e), lo);
            }
            fence_async();
            arrive_warp(bar(s.b.w_ready));
        }
    }
}

// ---------------------------------------------------------------- the mask's warpgroup

__device__ __forceinline__ void mask_role(const Launch &L, Shared &s, uint32_t tm, int i) {
    const gdn_linear &g = L.a.g;
    const int lane = i & 31, b = i >> 5;
    long long at = blockIdx.x;
    Unit x;
    uint32_t it = 0;
    while (next_unit(L, false, at, x)) {
        float gi = log_decay(g, x, 0, i);
        for (int c = 0; c < x.n; ++c, ++it) {
            const uint32_t slot = it & 1, half = (it >> 1) & 1;
            const uint32_t ts = tm + kScores + slot * 128 + ((uint32_t)b << 21);  // this warp's lanes
            const float lam = expf(gi);
            if (c + 1 < x.n) gi = log_decay(g, x, c + 1, i);
            if (!wait(bar(s.b.dec_full[slot]), half, &s.dead)) return;
            if (!wait(bar(s.b.s_full[slot]), half, &s.dead)) return;
            fence_after();
            const float rowf = s.rowf[slot][i];
            // Earlier 32s: all of their rows are seen.
#pragma unroll 1
            for (int m = 0; m < b; ++m) {
                float f = rowf;
                for (int k = m + 1; k < b; ++k) f *= s.t[slot][k];
                const float2 f2 = make_float2(f, f);
                uint32_t y[32];
                tmem_ld32(ts + 32 * m, y);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float4 cf = *reinterpret_cast<const float4 *>(&s.cf[slot][32 * m + e]);
                    const float2 p0 = mul2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])),
                                           mul2(make_float2(cf.x, cf.y), f2));
                    const float2 p1 = mul2(make_float2(__uint_as_float(y[e + 2]), __uint_as_float(y[e + 3])),
                                           mul2(make_float2(cf.z, cf.w), f2));
                    y[e / 2] = pack_bf16(p0.x, p0.y);
                    y[e / 2 + 1] = pack_bf16(p1.x, p1.y);
                }
                tmem_st16(ts + 16 * m, y);  // over scores that have been read
            }
            // The row's own 32, up to itself.
            {
                uint32_t y[32];
                tmem_ld32(ts + 32 * b, y);
                wait_ld();
                float d = 1.f;
#pragma unroll
                for (int e = 31; e >= 0; --e) {
                    if (e < 31) {
                        const float next = __shfl_sync(0xffffffffu, lam, e + 1);
                        if (e + 1 <= lane) d *= next;
                    }
                    y[e] = e <= lane ? __float_as_uint(__uint_as_float(y[e]) * d) : 0u;
                }
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    y[e / 2] = pack_bf16(__uint_as_float(y[e]), __uint_as_float(y[e + 1]));
                tmem_st16(ts + 16 * b, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = 0u;
#pragma unroll 1
                for (int m = b + 1; m < 4; ++m) tmem_st16(ts + 16 * m, y);
            }
            arrive_warp(bar(s.b.dec_empty[slot]));
            wait_st();
            fence_before();
            arrive_warp(bar(s.b.p_ready[slot]));
        }
    }
}

// ---------------------------------------------------------------- the state's warpgroup

template <bool OUT, bool STATE>
__device__ __forceinline__ void state_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm, int d) {
    const gdn_linear &g = L.a.g;
    const uint32_t tu = tm + kU + ((uint32_t)(d >> 5) << 21);
    long long at = blockIdx.x;
    Unit x;
    uint32_t it = 0;
    while (next_unit(L, !OUT, at, x)) {
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
        for (int c = 0; c < x.n; ++c, ++it) {
            const uint32_t slot = it & 1, half = (it >> 1) & 1;
            if (OUT) {
                if (!wait(bar(s.b.st_free), (it & 1) ^ 1, &s.dead)) return;
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
            if (!wait(bar(s.b.dec_full[slot]), half, &s.dead)) return;
            const float keep = s.t[slot][0] * s.t[slot][1] * (s.t[slot][2] * s.t[slot][3]);
            arrive_warp(bar(s.b.dec_empty[slot]));
            if (!wait(bar(s.b.u_full[slot]), half, &s.dead)) return;
            fence_after();
#pragma unroll
            for (int e = 0; e < NV; e += 16) {
                uint32_t y[16];
                tmem_ld16(tu + slot * NV + e, y);
                wait_ld();
#pragma unroll
                for (int m = 0; m < 16; m += 2) {
                    const float2 z = fma2(make_float2(S[e + m], S[e + m + 1]), make_float2(keep, keep),
                                          make_float2(__uint_as_float(y[m]), __uint_as_float(y[m + 1])));
                    S[e + m] = z.x;
                    S[e + m + 1] = z.y;
                }
            }
            fence_before();
            arrive_warp(bar(s.b.u_free[slot]));
        }
        if (STATE && d < g.dk) {
#pragma unroll
            for (int e = 0; e < NV; e += 4)
                __stcs(reinterpret_cast<float4 *>(row + e), make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]));
        }
    }
}

// ---------------------------------------------------------------- the output's warpgroup

__device__ __forceinline__ void output_role(const Launch &L, Shared &s, const Tiles &t, uint32_t tm, int i) {
    const gdn_linear &g = L.a.g;
    const int lane = i & 31, b = i >> 5;
    const uint32_t lanes = (uint32_t)b << 21;
    long long at = blockIdx.x;
    Unit x;
    uint32_t it = 0, stored = 0;
    while (next_unit(L, false, at, x)) {
        for (int c = 0; c < x.n; ++c, ++it) {
            const uint32_t slot = it & 1, half = (it >> 1) & 1;
            const int n = min(C, x.u.T - c * C);
            if (!wait(bar(s.b.dec_full[slot]), half, &s.dead)) return;
            float f = s.rowf[slot][i] * g.scale;
            for (int m = 0; m < b; ++m) f *= s.t[slot][m];
            arrive_warp(bar(s.b.dec_empty[slot]));
            if (!wait(bar(s.b.o_full), it & 1, &s.dead)) return;
            fence_after();
            // The block's queries have been read: its output goes through their place.
            const uint32_t stage = t.q + slot * kKeyTile;
            const float2 f2 = make_float2(f, f), scale2 = make_float2(g.scale, g.scale);
#pragma unroll
            for (int h = 0; h < NV; h += 32) {
                uint32_t y[32], z[32];
                tmem_ld32(tm + kO1 + lanes + h, y);
                tmem_ld32(tm + kO2 + lanes + h, z);
                wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float2 p = fma2(make_float2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])), f2,
                                          mul2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), scale2));
                    y[e / 2] = pack_bf16(p.x, p.y);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) sts128(chunk(stage, i, h / 8 + e), y + 4 * e);
            }
            fence_before();
            arrive_warp(bar(s.b.o_free));
            const int row = x.u.row0 + c * C, col = x.h * g.dv + x.c0;
            if (n == C) {
                fence_async();
                arrive_warp(bar(s.b.o_sync));
                if (b == 0) {
                    if (!wait(bar(s.b.o_sync), stored & 1, &s.dead)) return;
                    if (lane == 0) {
                        tma_store(&L.o, col, row, stage);
                        asm volatile("cp.async.bulk.commit_group;\ncp.async.bulk.wait_group.read 0;\n" ::: "memory");
                    }
                }
                ++stored;
            } else {
                __syncwarp();
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(L.a.o) + col + (lane & 7) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int r = 32 * b + 4 * e + (lane >> 3);
                    uint32_t y[4];
                    lds128(chunk(stage, r, lane & 7), y);
                    if (r < n)
                        *reinterpret_cast<uint4 *>(o + (long long)(row + r) * g.heads * g.dv) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_async();  // before the copy that follows into the same place
            }
            arrive_warp(bar(s.b.q_empty[slot]));
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
            mbar_init(bar(s.b.k_full[i]), 1);
            mbar_init(bar(s.b.v_full[i]), 1);
            mbar_init(bar(s.b.q_empty[i]), 4);
            mbar_init(bar(s.b.k_empty[i]), 1);
            mbar_init(bar(s.b.v_empty[i]), 1);
            mbar_init(bar(s.b.dec_full[i]), 4);
            mbar_init(bar(s.b.dec_empty[i]), OUT ? 12 : 4);
            mbar_init(bar(s.b.s_full[i]), 1);
            mbar_init(bar(s.b.p_ready[i]), 4);
            mbar_init(bar(s.b.u_full[i]), 1);
            mbar_init(bar(s.b.u_free[i]), 4);
        }
        mbar_init(bar(s.b.w_ready), 4);
        mbar_init(bar(s.b.w_free), 1);
        mbar_init(bar(s.b.st_ready), 4);
        mbar_init(bar(s.b.st_free), 1);
        mbar_init(bar(s.b.o_full), 1);
        mbar_init(bar(s.b.o_free), 4);
        mbar_init(bar(s.b.w_sync), 4);
        mbar_init(bar(s.b.o_sync), 4);
        mbar_init(bar(s.b.drain), 1);
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
            if (tid == 384) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
        }
    } else if (warp == 16) {
        if ((tid & 31) == 0) {
            uint32_t issued = 0;
            load_role<OUT>(L, s, t, issued);
            // Every copy has landed before the block ends (its roles waited for them unless one gave up).
            for (uint32_t p = issued > 2 ? issued - 2 : 0; s.dead && p <= issued; ++p) {
                wait_parity(bar(s.b.v_full[p & 1]), (p >> 1) & 1);
                wait_parity(bar(s.b.k_full[p & 1]), (p >> 1) & 1);
                if (OUT) wait_parity(bar(s.b.q_full[p & 1]), (p >> 1) & 1);
            }
        }
    } else {
        mma_role<OUT>(L, s, t, tm);
        commit(elect(), bar(s.b.drain));
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

// Rows of `cols` elements, `stride` apart; boxes of 64 columns by a block's rows.  Rows past the end
// read as zeros.
bool encode_rows(CUtensorMap *map, const void *base, long long cols, long long rows, long long stride) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t box[2] = {64, C};
    const cuuint32_t elem[2] = {1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                     elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t launch_tc(const LinearArgs &a, cudaStream_t stream) {
    const gdn_linear &g = a.g;
    Launch L;
    L.a = a;
    L.slices = g.dv / NV;
    L.units = (long long)g.batch * g.heads * L.slices;
    const long long krow = (long long)g.k_heads * g.dk, vrow = (long long)g.heads * g.dv;
    if (!encoder() || !encode_rows(&L.k, g.k, krow, g.n_tok, g.k_stride) ||
        !encode_rows(&L.v, g.v, vrow, g.n_tok, g.v_stride))
        return cudaErrorInvalidValue;
    L.q = L.k;  // not used by a commit
    L.o = L.v;
    if (MODE != kCommit && (!encode_rows(&L.q, g.q, krow, g.n_tok, g.q_stride) ||
                            !encode_rows(&L.o, a.o, vrow, g.n_tok, vrow)))
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
