// Attention over a paged cache for few query rows a key head (bf16): single
// tokens and short drafts.
//
// Bound by the cache's bytes: 16 rows use each key and value once, 16 flops a
// byte.  So the kernel is a stream of the cache through shared memory with the
// products beside it.  A block is a few warps; a key tile is 16 places a warp,
// and each warp is a stream of its own: it copies its places' keys and values
// (cp.async, 16-byte chunks XOR-swizzled by row, a ring of tiles ahead), and
// keeps its own running maximum, total and output for all 16 rows, so that
// nothing in the loop waits for another warp.  The warps' results are joined
// through shared memory at the end of a segment; the partials of a unit that
// spans blocks by the block that writes the last one, or by combine_kernel where
// there may be many.  Two blocks an SM: one streams while the other joins.
//
// The products are mma.sync m16n8k16: 16 rows fill its M, where a 128-row
// tcgen05 tile would be seven eighths padding, and the fragments of the scores
// are those of the weights, so nothing goes through memory in between.  The
// weights enter the second product as two bf16 terms (w = hi + lo, 2^-16 w
// left): the tensor cores have the time while the cache streams, and the result
// is then as exact as one with float32 weights (error against 64 bits 0.0017, that of the
// rounded output alone).  hi is w cut off, so that lo is not negative, and lo of a weight
// that is not zero is kept above zero: both terms of an infinite value then have its sign.
//
// Measured: 64 requests' single tokens over contexts of up to 8191 places, 8 key heads
// of 128: 1.33 GB in 203 to 207 us, 6.4 TB/s, 95% of a plain copy's rate, with the tensor pipe
// 28% and the issue slots 31% busy.  2 key heads of 256: 0.66 GB in 120 us.  More rows than 16 read
// the cache once for each 16 of them (heads of 32 and 256 have no other kernel): 16 drafts of
// 8 heads each over up to 4000 places 433 us, where the bytes would take 50.  A single request's token over 1000 places 11 us:
// latencies in a row (lengths, pages, keys, the join of the workers).
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kRows = 16;
constexpr int kAlign = 16;  // a warp's places: within one page
constexpr int kExtra = 1;   // a unit's start and end, in tiles

template <int HD>
struct Cfg {
    static constexpr int W = HD == 256 ? 2 : 4;        // warps
    static constexpr int S = HD == 256 ? 2 : HD == 128 ? 3 : HD == 64 ? 6 : 8;  // tiles of the ring
    static constexpr int KT = 16 * W;                  // places of a block's tile
    static constexpr int NT = 32 * W;
    static constexpr int kTile = 16 * HD * 2;          // bytes of a warp's keys (or values)
    static constexpr bool kQInSmem = HD == 256;        // else in registers
    static constexpr int kJoin = W / 2 * kRows * HD * 4;
    static constexpr int kSmem = W * S * 2 * kTile + kJoin + (kQInSmem ? kRows * HD * 2 : 0);
};

// Byte offset of 16-byte chunk c of row r in a tile of HD-element rows: eight rows
// of the same chunk lie in different banks.
template <int HD>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    const int x = HD >= 64 ? (r & 7) : ((r >> 1) & 3);
    return (uint32_t)(r * HD * 2 + ((c ^ x) << 4));
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

// 16 bytes, or zeros where !keep (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool keep) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
                 "r"(keep ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// The two bf16 terms of weights x, y >= 0 (or NaN).  lo is raised to 2^-126, of which no more
// than that part of a value is added; it stays 0 for a weight of 0.
__device__ __forceinline__ void split_weights(float x, float y, uint32_t &hi, uint32_t &lo) {
    constexpr float kTiny = 0x1p-126f;
    hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    lo = pack_bf16(fmaxf(x - __uint_as_float(hi << 16), fminf(x, kTiny)),
                   fmaxf(y - __uint_as_float(hi & 0xFFFF0000u), fminf(y, kTiny)));
}

// Whether one of the two bf16 is infinite or NaN.
__device__ __forceinline__ bool not_finite2(uint32_t x) {
    return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
}

// The page of a warp's 16 places of tile i, or -1 when no row sees one of them.
template <int HD>
__device__ __forceinline__ int page_of(const AttnArgs &a, const Segment &g, int i, int warp) {
    const int v0 = i * Cfg<HD>::KT + warp * 16;
    if (!some_see(a, g.span, v0, v0 + 15)) return -1;
    return a.page_table[(long long)g.r * a.max_pages + (place_of(g.span, v0) >> a.page_shift)];
}

// Copies a warp's 16 places of tile i of segment g, in `page`, into its ring slot.
template <int HD>
__device__ __forceinline__ void copy_tile(const AttnArgs &a, const Segment &g, int i, int page, int warp,
                                          int lane, uint32_t kdst) {
    using C = Cfg<HD>;
    const int v0 = i * C::KT + warp * 16;
    const TileSpan &sp = g.span;
    if (!some_see(a, sp, v0, v0 + 15)) return;
    const int j0 = place_of(sp, v0);
    const bool page_ok = page >= 0 && page < a.n_pages;
    if (!page_ok && lane == 0 && a.dev_err) atomicOr(a.dev_err, GDN_DEVERR_PAGE);
    const long long at = page_ok ? (long long)page * a.page_stride +
                                       (((long long)g.h << a.page_shift) +
                                        (j0 & ((1 << a.page_shift) - 1))) * HD
                                 : 0;
    const char *kp = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(a.k) + at);
    const char *vp = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(a.v) + at);
    constexpr int CR = HD / 8;  // chunks of a row
    // a place that no row sees may hold anything: it is zeros here
    const bool each = v0 + 15 <= sp.pmax && (a.window == 0 || v0 > sp.pmin - a.window || v0 + 15 < sp.sinks);
    auto copy = [&](auto keep) {
#pragma unroll
        for (int u = 0; u < CR / 2; ++u) {
            const int x = u * 32 + lane, r = x / CR, c = x % CR;
            const bool k = keep(r);
            copy16(kdst + chunk_at<HD>(r, c), kp + (k ? x * 16 : 0), k);
            copy16(kdst + C::kTile + chunk_at<HD>(r, c), vp + (k ? x * 16 : 0), k);
        }
    };
    if (each && page_ok)
        copy([](int) { return true; });
    else
        copy([&](int r) { return page_ok && some_see(a, sp, v0 + r, v0 + r); });
}

template <int HD>
__global__ void __launch_bounds__(Cfg<HD>::NT, 2) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
    using C = Cfg<HD>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ PlanScratch plan;
    __shared__ float top[C::W][kRows], sum[C::W][kRows];
    __shared__ int2 joined;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = blockIdx.x, P = gridDim.x;
    float *join = reinterpret_cast<float *>(smem + C::W * C::S * 2 * C::kTile);
    unsigned char *qs = smem + C::W * C::S * 2 * C::kTile + C::kJoin;
    const uint32_t ring = smem_addr(smem) + warp * C::S * 2 * C::kTile;

    // Two cursors over the same segments: the copies run S - 1 tiles ahead of the products,
    // across segments of any length, with one group a tile.
    Cursor cur = make_plan<C::NT, kRows, C::KT, kExtra, 2>(a, c, P, kAlign, &plan, c == 0);
    Cursor in = cur;
    Segment g, gi;        // in use, and being copied
    int ia = 0, ia_end = 0, page = 0;  // tile to copy next, and the page it lies in
    int slot_in = 0, slot_out = 0;
    auto advance = [&]() {  // one more tile on its way; at the end of the range an empty group
        if (ia >= ia_end && next_segment<kRows, C::KT, kExtra>(a, kAlign, in, gi)) {
            ia = gi.i0;
            ia_end = gi.i1;
            page = page_of<HD>(a, gi, ia, warp);
        }
        if (ia < ia_end) {
            const int here = page;
            if (ia + 1 < ia_end) page = page_of<HD>(a, gi, ia + 1, warp);  // a tile ahead
            copy_tile<HD>(a, gi, ia++, here, warp, lane, ring + slot_in * 2 * C::kTile);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
        slot_in = slot_in + 1 == C::S ? 0 : slot_in + 1;
    };
#pragma unroll 1
    for (int s = 0; s < C::S - 1; ++s) advance();

    // Fragment coordinates: rows qr and qr + 8, columns 2 qc, 2 qc + 1 of 8.
    const int qr = lane >> 2, qc = lane & 3;
    bool any = false;
    while (next_segment<kRows, C::KT, kExtra>(a, kAlign, cur, g)) {
        any = true;
        const int rows = min(kRows, g.req.T * a.G - g.qt * kRows);
        const TileSpan sp = g.span;
        int own[2];  // the rows' own places, as numbered in the span
        const __nv_bfloat16 *qrow[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = g.qt * kRows + qr + 8 * e, t = div_group(a, i);
            own[e] = g.req.ctx + t - sp.shift;
            qrow[e] = static_cast<const __nv_bfloat16 *>(a.q) + (g.req.row0 + t) * a.q_stride +
                      (g.h * a.G + i - t * a.G) * HD;
        }
        const bool has[2] = {qr < rows, qr + 8 < rows};
        uint32_t qf[C::kQInSmem ? 1 : HD / 16][4];
        if constexpr (C::kQInSmem) {
            __syncthreads();  // the previous segment's queries are no longer read
            for (int x = tid; x < kRows * (HD / 8); x += C::NT) {
                const int r = x / (HD / 8), ch = x % (HD / 8), i = g.qt * kRows + r;
                const int t = div_group(a, i);
                uint4 w = make_uint4(0, 0, 0, 0);
                if (r < rows)
                    w = *reinterpret_cast<const uint4 *>(
                        static_cast<const __nv_bfloat16 *>(a.q) + (g.req.row0 + t) * a.q_stride +
                        (g.h * a.G + i - t * a.G) * HD + ch * 8);
                *reinterpret_cast<uint4 *>(qs + chunk_at<HD>(r, ch)) = w;
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qf[k][e] = has[e & 1] ? *reinterpret_cast<const uint32_t *>(
                                                qrow[e & 1] + k * 16 + (e >> 1) * 8 + qc * 2)
                                          : 0u;
        }
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[HD / 8][4];
#pragma unroll
        for (int n = 0; n < HD / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

        for (int i = g.i0; i < g.i1; ++i) {
            // No branch around this wait: the group's copies would be waited for one and all.
            asm volatile("cp.async.wait_group %0;\n" ::"n"(C::S - 2) : "memory");
            __syncwarp();
            advance();
            const uint32_t kt = ring + slot_out * 2 * C::kTile, vt = kt + C::kTile;
            slot_out = slot_out + 1 == C::S ? 0 : slot_out + 1;
            const int v0 = i * C::KT + warp * 16;
            if (!some_see(a, sp, v0, v0 + 15)) continue;
            float s[2][4] = {};
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                uint32_t b[4];
                ldsm4(b, kt + chunk_at<HD>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                if constexpr (C::kQInSmem) {
                    uint32_t qa[4];
                    ldsm4(qa, smem_addr(qs) + chunk_at<HD>(lane & 15, 2 * k + (lane >> 4)));
                    mma16816(s[0], qa, b[0], b[1]);
                    mma16816(s[1], qa, b[2], b[3]);
                } else {
                    mma16816(s[0], qf[k], b[0], b[1]);
                    mma16816(s[1], qf[k], b[2], b[3]);
                }
            }
            // Every row sees all 16 places, or some are hidden from some rows.
            const bool full = all_see(a, sp, v0, v0 + 15);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] *= a.scale_log2;
                    if (!full && !row_sees(a, sp, own[e >> 1], v0 + n * 8 + qc * 2 + (e & 1)))
                        s[n][e] = -INFINITY;
                }
            float mn[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                mn[e] = fmaxf(m[e], x);
            }
            if (__any_sync(0xffffffffu, mn[0] != m[0] || mn[1] != m[1])) {
                // a new maximum: rarer and rarer along the cache
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    keep[e] = mn[e] == -INFINITY ? 0.f : exp2_fast(m[e] - mn[e]);
                    m[e] = mn[e];
                    l[e] *= keep[e];
                }
#pragma unroll
                for (int n = 0; n < HD / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] *= keep[e >> 1];
            }
            const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = exp2_fast(s[n][e] - base[e >> 1]);
                    l[e >> 1] += s[n][e];
                }
            // Where some rows must not see a value that is not finite, a product with
            // its zero weight would still be NaN: such tiles are added value by value, to the rows
            // that see it.
            bool odd = false;
            if (!full) {
#pragma unroll
                for (int n = 0; n < HD / 16; ++n) {
                    uint32_t b[4];
                    ldsm4t(b, vt + chunk_at<HD>(lane & 15, 2 * n + (lane >> 4)));
                    odd |= not_finite2(b[0]) || not_finite2(b[1]) || not_finite2(b[2]) || not_finite2(b[3]);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (!odd) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    split_weights(s[e >> 1][(e & 1) * 2], s[e >> 1][(e & 1) * 2 + 1], hi[e], lo[e]);
#pragma unroll
                for (int n = 0; n < HD / 16; ++n) {
                    uint32_t b[4];
                    ldsm4t(b, vt + chunk_at<HD>(lane & 15, 2 * n + (lane >> 4)));
                    mma16816(o[2 * n], hi, b[0], b[1]);
                    mma16816(o[2 * n + 1], hi, b[2], b[3]);
                    mma16816(o[2 * n], lo, b[0], b[1]);
                    mma16816(o[2 * n + 1], lo, b[2], b[3]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int from = (lane & ~3) | ((j & 7) >> 1);
                    const float p0 = __shfl_sync(0xffffffffu, s[j >> 3][j & 1], from);
                    const float p1 = __shfl_sync(0xffffffffu, s[j >> 3][2 + (j & 1)], from);
                    const bool adds[2] = {row_sees(a, sp, own[0], v0 + j), row_sees(a, sp, own[1], v0 + j)};
#pragma unroll
                    for (int n = 0; n < HD / 8; ++n) {
                        uint32_t v;
                        asm volatile("ld.shared.b32 %0, [%1];"
                                     : "=r"(v)
                                     : "r"(vt + chunk_at<HD>(j, n) + qc * 4)
                                     : "memory");
                        const float x = __uint_as_float(v << 16), y = __uint_as_float(v & 0xFFFF0000u);
                        if (adds[0]) {
                            o[n][0] = fmaf(p0, x, o[n][0]);
                            o[n][1] = fmaf(p0, y, o[n][1]);
                        }
                        if (adds[1]) {
                            o[n][2] = fmaf(p1, x, o[n][2]);
                            o[n][3] = fmaf(p1, y, o[n][3]);
                        }
                    }
                }
            }
        }

        // Join the warps: each scales its output to the block's maximum, then they are
        // added in pairs through shared memory.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (qc == 0) {
                top[warp][qr + 8 * e] = m[e];
                sum[warp][qr + 8 * e] = l[e];
            }
        }
        __syncthreads();
        float all[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x = top[0][qr + 8 * e];
#pragma unroll
            for (int w = 1; w < C::W; ++w) x = fmaxf(x, top[w][qr + 8 * e]);
            const float base = x == -INFINITY ? 0.f : x;
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < C::W; ++w)
                total = fmaf(sum[w][qr + 8 * e], exp2_fast(top[w][qr + 8 * e] - base), total);
            const float keep = exp2_fast(m[e] - base);
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
                o[n][2 * e] *= keep;
                o[n][2 * e + 1] *= keep;
            }
            m[e] = x;
            all[e] = total;
        }
#pragma unroll
        for (int half = C::W / 2; half >= 1; half /= 2) {
            if (warp >= half && warp < 2 * half) {
                float4 *dst = reinterpret_cast<float4 *>(join + (warp - half) * kRows * HD);
#pragma unroll
                for (int n = 0; n < HD / 8; ++n)
                    dst[n * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
            }
            __syncthreads();
            if (warp < half) {
                const float4 *src = reinterpret_cast<const float4 *>(join + warp * kRows * HD);
#pragma unroll
                for (int n = 0; n < HD / 8; ++n) {
                    const float4 x = src[n * 32 + lane];
                    o[n][0] += x.x;
                    o[n][1] += x.y;
                    o[n][2] += x.z;
                    o[n][3] += x.w;
                }
            }
            // the warps that read may be written over in the next round
            if (half > 1) __syncthreads();
        }
        if (warp == 0) {
            const bool whole = g.i0 == 0 && g.i1 == sp.n;
            float *part = a.part + (long long)part_slot(c, g) * kRows * (HD + 2);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (!has[e]) continue;
                const int row = qr + 8 * e, i = g.qt * kRows + row;
                if (whole) {
                    const int t = div_group(a, i);
                    const long long at = (long long)(g.req.row0 + t) * a.Hq + g.h * a.G + i - t * a.G;
                    const float inv = 1.f / all[e];
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.o) + at * HD + qc * 2;
#pragma unroll
                    for (int n = 0; n < HD / 8; ++n)
                        *reinterpret_cast<uint32_t *>(dst + n * 8) =
                            pack_bf16(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                    if (a.lse && qc == 0) a.lse[at] = (m[e] + log2f(all[e])) * 0.69314718055994531f;
                } else {
#pragma unroll
                    for (int n = 0; n < HD / 8; ++n)
                        *reinterpret_cast<float2 *>(part + part_at<kRows>(row, n * 8 + qc * 2)) =
                            make_float2(o[n][2 * e], o[n][2 * e + 1]);
                    if (qc == 0) {
                        part[kRows * HD + row] = m[e];
                        part[kRows * HD + kRows + row] = all[e];
                    }
                }
            }
        }
        if (a.count && !(g.i0 == 0 && g.i1 == sp.n))
            join_if_last<__nv_bfloat16, kRows, HD, C::NT>(a, c, g, cur.x, cur.N, cur.P, &joined);
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (tid == 0 && !a.count) write_desc(a, c, g, any, cur.x, cur.N, cur.P);
}

template <int HD>
cudaError_t launch_hd(const AttnArgs &a, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attn_rows_kernel<HD>>(Cfg<HD>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kAttnWorkers);
    cfg.blockDim = dim3(Cfg<HD>::NT);
    cfg.dynamicSmemBytes = Cfg<HD>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_rows_kernel<HD>, a);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t stream) {
    switch (a.hd) {
        case 32: return launch_hd<32>(a, stream);
        case 64: return launch_hd<64>(a, stream);
        case 128: return launch_hd<128>(a, stream);
        default: return launch_hd<256>(a, stream);
    }
}

}  // namespace gdn
