// Attention of a step's rows over a paged key/value cache: the CUDA-core
// kernel, and the kernel that joins partial results.
//
// The softmax runs in one pass over the keys with a running maximum m and
// total l per row, in powers of two: with x_j = scale log2(e) q.k_j,
//     m' = max(m, max_j x_j),  l' = l 2^(m - m') + sum_j 2^(x_j - m'),
//     o' = o 2^(m - m') + sum_j 2^(x_j - m') v_j,
// and o / l at the end.  m = -inf (no key seen yet) is replaced by 0 in the
// exponents, so a row whose mask hides a whole tile, or a whole worker's
// range, adds nothing instead of NaN.
#include <algorithm>
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kRows = 16;   // query rows of a unit
constexpr int kKeys = 32;   // places of a key tile
constexpr int kThreads = 128;
constexpr int kAlign = 16;  // pages begin at multiples of it
constexpr int kMaxParts = 48;  // joined by one block; more by a launch of their own
constexpr int kMinTiles = 2;
constexpr int kExtra = 1;   // a unit's start and end, in tiles

template <int HD>
struct Smem {
    static constexpr int LD = HD + 4;  // rows 16-byte aligned, 4 banks apart
    float q[kRows][LD];
    float k[kKeys][LD];
    float v[kKeys][LD];
    float p[kRows][kKeys + 1];
    PlanScratch plan;
    int2 join;
};

// 16 bytes of a row -> floats in shared memory.
template <typename T>
__device__ __forceinline__ void put_vec(float *dst, const uint4 &w) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4 *>(dst) = w;
    } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dst[2 * e] = __uint_as_float(x[e] << 16);
            dst[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
        }
    }
}

// Thread (row = tid / 8, sub = tid % 8) of the block: scores of keys sub + 8 i,
// output columns 4 sub + 32 i.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreads) attn_simple_kernel(const __grid_constant__ AttnArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<HD> &s = *reinterpret_cast<Smem<HD> *>(raw);
    constexpr int VE = 16 / (int)sizeof(T), VR = HD / VE;  // vectors of a row
    const int tid = threadIdx.x, c = blockIdx.x, P = gridDim.x;
    const int row = tid >> 3, sub = tid & 7;
    Cursor cur = make_plan<kThreads, kRows, kKeys, kExtra, kMinTiles>(a, c, P, kAlign, &s.plan, c == 0);
    Segment g;
    bool any = false;
    while (next_segment<kRows, kKeys, kExtra>(a, kAlign, cur, g)) {
        any = true;
        __syncthreads();  // the previous segment's tiles are no longer read
        const int rows = min(kRows, g.req.T * a.G - g.qt * kRows);
        for (int i = tid; i < kRows * VR; i += kThreads) {
            const int ri = i / VR, e = i % VR * VE;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (ri < rows) {
                const int t = (g.qt * kRows + ri) / a.G, gh = (g.qt * kRows + ri) % a.G;
                w = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.q) +
                                                     (g.req.row0 + t) * a.q_stride +
                                                     (g.h * a.G + gh) * HD + e);
            }
            put_vec<T>(&s.q[ri][e], w);
        }
        // this thread's row's own place, as numbered in the span
        const int own = g.req.ctx + (g.qt * kRows + row) / a.G - g.span.shift;
        float m = -INFINITY, l = 0.f, o[HD / 8] = {};
        for (int i = g.i0; i < g.i1; ++i) {
            const int v0 = i * kKeys;
            __syncthreads();
            for (int x = tid; x < kKeys * VR; x += kThreads) {
                const int kj = x / VR, e = x % VR * VE, j = place_of(g.span, v0 + kj);
                uint4 wk = make_uint4(0, 0, 0, 0), wv = wk;
                if (some_see(a, g.span, v0 + kj, v0 + kj)) {
                    const int page =
                        a.page_table[(long long)g.r * a.max_pages + (j >> a.page_shift)];
                    if (page >= 0 && page < a.n_pages) {
                        const long long at =
                            (long long)page * a.page_stride +
                            (((long long)g.h << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * HD + e;
                        wk = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.k) + at);
                        wv = *reinterpret_cast<const uint4 *>(static_cast<const T *>(a.v) + at);
                    } else if (a.dev_err) {
                        atomicOr(a.dev_err, GDN_DEVERR_PAGE);
                    }
                }
                put_vec<T>(&s.k[kj][e], wk);
                put_vec<T>(&s.v[kj][e], wv);
            }
            __syncthreads();
            float x[kKeys / 8] = {};
#pragma unroll 4
            for (int e = 0; e < HD; e += 4) {
                const float4 qv = *reinterpret_cast<const float4 *>(&s.q[row][e]);
#pragma unroll
                for (int u = 0; u < kKeys / 8; ++u) {
                    const float4 kv = *reinterpret_cast<const float4 *>(&s.k[sub + 8 * u][e]);
                    x[u] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, x[u]))));
                }
            }
            float top = -INFINITY;
            bool seen[kKeys / 8];
#pragma unroll
            for (int u = 0; u < kKeys / 8; ++u) {
                seen[u] = row < rows && row_sees(a, g.span, own, v0 + sub + 8 * u);
                x[u] = seen[u] ? x[u] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, x[u]);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
            const float keep = exp2f(m - base);  // 0 while m = -inf
            float part = 0.f;
#pragma unroll
            for (int u = 0; u < kKeys / 8; ++u) {
                const float e = exp2f(x[u] - base);
                s.p[row][sub + 8 * u] = seen[u] ? e : 0.f;
                part += seen[u] ? e : 0.f;
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
            l = l * keep + part;
            m = mn;
#pragma unroll
            for (int u = 0; u < HD / 8; ++u) o[u] *= keep;
            __syncwarp();  // the row's scores come from threads of this warp only
            for (int kj = 0; kj < kKeys; ++kj) {
                const float p = s.p[row][kj];
                if (p == 0.f) continue;  // a hidden place adds nothing, whatever v holds there
#pragma unroll
                for (int u = 0; u < HD / 32; ++u) {
                    const float4 vv = *reinterpret_cast<const float4 *>(&s.v[kj][4 * sub + 32 * u]);
                    o[4 * u] = fmaf(p, vv.x, o[4 * u]);
                    o[4 * u + 1] = fmaf(p, vv.y, o[4 * u + 1]);
                    o[4 * u + 2] = fmaf(p, vv.z, o[4 * u + 2]);
                    o[4 * u + 3] = fmaf(p, vv.w, o[4 * u + 3]);
                }
            }
            __syncwarp();
        }
        if (row < rows) {
            if (g.i0 == 0 && g.i1 == g.span.n) {
                const int t = (g.qt * kRows + row) / a.G, gh = (g.qt * kRows + row) % a.G;
                const long long at = (long long)(g.req.row0 + t) * a.Hq + g.h * a.G + gh;
                const float inv = 1.f / l;
#pragma unroll
                for (int u = 0; u < HD / 8; u += 4)
                    put(static_cast<T *>(a.o) + at * HD + 4 * sub + 8 * u,
                        make_float4(o[u] * inv, o[u + 1] * inv, o[u + 2] * inv, o[u + 3] * inv));
                if (a.lse && sub == 0) a.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
            } else {
                float *dst = a.part + (long long)part_slot(c, g) * kRows * (HD + 2);
#pragma unroll
                for (int u = 0; u < HD / 8; u += 4)
                    *reinterpret_cast<float4 *>(dst + part_at<kRows>(row, 4 * sub + 8 * u)) =
                        make_float4(o[u], o[u + 1], o[u + 2], o[u + 3]);
                if (sub == 0) {
                    dst[kRows * HD + row] = m;
                    dst[kRows * HD + kRows + row] = l;
                }
            }
        }
        if (a.count && !(g.i0 == 0 && g.i1 == g.span.n))
            join_if_last<T, kRows, HD, kThreads>(a, c, g, cur.x, cur.N, cur.P, &s.join);
    }
    if (tid == 0 && !a.count) write_desc(a, c, g, any, cur.x, cur.N, cur.P);
}

// Joins the partials of a unit that spans workers c .. last: block (c, y) the eight rows and
// CGB column groups (of four) that y names, eight rows of a group being a line.  SLICES
// threads share a value's partials, added in the order of the workers and then of the
// slices.
template <int ROWS, int HD>
struct Combine {
    static constexpr int CG = HD / 4;
    static constexpr int kWant = ROWS == 16 ? 8 : ROWS == 128 ? 16 : 32;
    static constexpr int CGB = CG < kWant ? CG : kWant;
    static constexpr int SLICES = 256 / (8 * CGB);
    static constexpr int kBlocks = ROWS / 8 * (CG / CGB);
};

template <typename T, int ROWS, int HD>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnArgs a) {
    using C = Combine<ROWS, HD>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Partial<1> part[C::SLICES][8 * C::CGB];
    const int c = blockIdx.x;
    const int4 d0 = a.desc[2 * c], d1 = a.desc[2 * c + 1];
    const int last = d0.x, qt = d0.y, h = d0.z, row0 = d0.w, T_r = d1.x;
    const int rb = (int)blockIdx.y / (C::CG / C::CGB) * 8, cb = blockIdx.y % (C::CG / C::CGB) * C::CGB;
    if (last < 0 || qt * ROWS + rb >= T_r * a.G) return;
    const int item = threadIdx.x % (8 * C::CGB), slice = threadIdx.x / (8 * C::CGB);
    const int row = rb + (item & 7), cg = cb + (item >> 3), i = qt * ROWS + row;
    Partial<1> s;
    add_partials<ROWS, HD, 1, 1>(a, s, c, c + slice, C::SLICES, last, row, cg);
    if (C::SLICES > 1) {
        if (slice > 0) part[slice][item] = s;
        __syncthreads();
        if (slice > 0) return;
#pragma unroll
        for (int k = 1; k < C::SLICES; ++k) s.add(part[k][item].m, part[k][item].l, part[k][item].o);
    }
    if (i >= T_r * a.G) return;
    const int t = div_group(a, i);
    const long long at = (long long)(row0 + t) * a.Hq + h * a.G + (i - t * a.G);
    const float inv = 1.f / s.l;
    put(static_cast<T *>(a.o) + at * HD + 4 * cg,
        make_float4(s.o[0].x * inv, s.o[0].y * inv, s.o[0].z * inv, s.o[0].w * inv));
    if (a.lse && cg == 0) a.lse[at] = (s.m + log2f(s.l)) * 0.69314718055994531f;
}

template <typename K>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, const AttnArgs &a,
                   cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int HD>
cudaError_t launch_simple(const AttnArgs &a, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attn_simple_kernel<float, HD>>((int)sizeof(Smem<HD>));
    if (e != cudaSuccess) return e;
    return launch(attn_simple_kernel<float, HD>, dim3(kAttnWorkers), kThreads, sizeof(Smem<HD>), a,
                  stream);
}

// The two launches of a call: finished units and partials, then the join.
template <int HD>
cudaError_t launch_hd(const AttnArgs &a, bool bf16, cudaStream_t stream) {
    const AttnKind kind = attn_kind(bf16, HD, (long long)a.max_T * a.G);
    const auto joined = [&](cudaError_t first, auto join, int workers, int blocks) {
        return first != cudaSuccess ? first
                                    : launch(join, dim3(workers, blocks), 256, 0, a, stream);
    };
    if constexpr (HD == 64 || HD == 128) {
        if (kind == kAttnDrafts)
            return joined(launch_attn_tc(a, false, stream), combine_kernel<__nv_bfloat16, 128, HD>,
                          kAttnTcWorkers, Combine<128, HD>::kBlocks);
        if (kind == kAttnWide)
            return joined(launch_attn_tc(a, true, stream), combine_kernel<__nv_bfloat16, 256, HD>,
                          kAttnTcWorkers, Combine<256, HD>::kBlocks);
    }
    const cudaError_t e = kind == kAttnSimple ? launch_simple<HD>(a, stream) : launch_attn_rows(a, stream);
    if (a.count) return e;
    return kind == kAttnSimple ? joined(e, combine_kernel<float, 16, HD>, kAttnWorkers,
                                        Combine<16, HD>::kBlocks)
                               : joined(e, combine_kernel<__nv_bfloat16, 16, HD>, kAttnWorkers,
                                        Combine<16, HD>::kBlocks);
}

}  // namespace

cudaError_t launch_attn(AttnArgs a, bool bf16, cudaStream_t stream) {
    // Few partials to a unit: the block that writes the last one joins them, and the second
    // launch is saved.  A request's key heads have equal work, so a unit spans at most
    // workers / key heads (and a bit) of them, and no more than its tiles allow.
    const AttnKind kind = attn_kind(bf16, a.hd, (long long)a.max_T * a.G);
    const long long tiles = ((long long)a.max_pages << a.page_shift) / 32;
    const long long parts = std::min<long long>(kAttnWorkers / a.Hkv, tiles / 2) + 2;
    if (kind == kAttnDrafts || kind == kAttnWide || parts > kMaxParts) a.count = nullptr;
    switch (a.hd) {
        case 32: return launch_hd<32>(a, bf16, stream);
        case 64: return launch_hd<64>(a, bf16, stream);
        case 128: return launch_hd<128>(a, bf16, stream);
        default: return launch_hd<256>(a, bf16, stream);
    }
}

// Which kernel runs, by type and rows a key head: float32 on the CUDA cores; up to
// 16 rows as one mma.sync tile; more on tcgen05, in units of 128 or 256 rows, for the
// heads whose tiles fit there.
AttnKind attn_kind(bool bf16, int hd, long long rows) {
    if (!bf16) return kAttnSimple;
    if (rows <= 16 || (hd != 64 && hd != 128)) return kAttnRows;
    return rows <= 128 ? kAttnDrafts : kAttnWide;
}

int64_t attn_workspace(bool bf16, int hd, long long rows) {
    const AttnKind kind = attn_kind(bf16, hd, rows);
    const int64_t workers = kind == kAttnDrafts || kind == kAttnWide ? kAttnTcWorkers : kAttnWorkers;
    const int64_t unit = kind == kAttnWide ? 256 : kind == kAttnDrafts ? 128 : 16;
    return kAttnHeader +
           2 * workers * unit * (hd + 2) * (int64_t)sizeof(float);
}

}  // namespace gdn
