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
constexpr int kThreads = 256;
constexpr int kLanes = kThreads / kRows;  // threads a row
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

// float32.  Thread (row = tid / 16, sub = tid % 16) of the block: the scores of keys sub
// and sub + 16, the output columns 4 sub + 64 u.  Bound by shared memory's reads: a float4 of
// queries and two of keys for eight products.  A tile is on its way to registers while the
// one before it is used.  Five requests of up to 7 rows over 777 places, 3 key heads of 64
// with 5 queries each: 16.5 us, of which the lengths, the pages and the join are most (4.7 MB
// read, FMA pipe 14% busy); with 128 threads and no tile ahead 18.2.
template <int HD>
__global__ void __launch_bounds__(kThreads) attn_simple_kernel(const __grid_constant__ AttnArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<HD> &s = *reinterpret_cast<Smem<HD> *>(raw);
    constexpr int VR = HD / 4;                         // vectors of a row
    constexpr int PER = kKeys * VR / kThreads;         // of a tile's keys (values) a thread
    constexpr int NC = HD >= 64 ? 4 : 2;               // neighbouring output columns of a thread
    constexpr int NO = HD / kLanes;                    // its output columns
    const int tid = threadIdx.x, c = blockIdx.x, P = gridDim.x;
    const int row = tid / kLanes, sub = tid % kLanes;
    Cursor cur = make_plan<kThreads, kRows, kKeys, kExtra, kMinTiles>(a, c, P, kAlign, &s.plan, c == 0);
    Segment g;
    bool any = false;
    while (next_segment<kRows, kKeys, kExtra>(a, kAlign, cur, g)) {
        any = true;
        uint4 wk[PER], wv[PER];
        auto fetch = [&](int i) {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int x = tid + u * kThreads, kj = x / VR, e = x % VR * 4;
                const int v = i * kKeys + kj, j = place_of(g.span, v);
                wk[u] = wv[u] = make_uint4(0, 0, 0, 0);
                if (!some_see(a, g.span, v, v)) continue;
                const int page = a.page_table[(long long)g.r * a.max_pages + (j >> a.page_shift)];
                if (page >= 0 && page < a.n_pages) {
                    const long long at =
                        (long long)page * a.page_stride +
                        (((long long)g.h << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * HD + e;
                    wk[u] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.k) + at);
                    wv[u] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.v) + at);
                } else if (a.dev_err) {
                    atomicOr(a.dev_err, GDN_DEVERR_PAGE);
                }
            }
        };
        fetch(g.i0);
        __syncthreads();  // the previous segment's tiles are no longer read
        const int rows = min(kRows, g.req.T * a.G - g.qt * kRows);
        for (int i = tid; i < kRows * VR; i += kThreads) {
            const int ri = i / VR, e = i % VR * 4, t = div_group(a, g.qt * kRows + ri);
            uint4 w = make_uint4(0, 0, 0, 0);
            if (ri < rows)
                w = *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) +
                                                     (g.req.row0 + t) * a.q_stride +
                                                     (g.h * a.G + g.qt * kRows + ri - t * a.G) * HD + e);
            *reinterpret_cast<uint4 *>(&s.q[ri][e]) = w;
        }
        // this thread's row's own place, as numbered in the span
        const int tok = div_group(a, g.qt * kRows + row);
        const int own = g.req.ctx + tok - g.span.shift;
        float m = -INFINITY, l = 0.f, o[NO] = {};
        for (int i = g.i0; i < g.i1; ++i) {
            const int v0 = i * kKeys;
            if (i > g.i0) __syncthreads();
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int x = tid + u * kThreads, kj = x / VR, e = x % VR * 4;
                *reinterpret_cast<uint4 *>(&s.k[kj][e]) = wk[u];
                *reinterpret_cast<uint4 *>(&s.v[kj][e]) = wv[u];
            }
            __syncthreads();
            if (i + 1 < g.i1) fetch(i + 1);
            float x[2] = {};
#pragma unroll 8
            for (int e = 0; e < HD; e += 4) {
                const float4 qv = *reinterpret_cast<const float4 *>(&s.q[row][e]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 kv = *reinterpret_cast<const float4 *>(&s.k[sub + kLanes * u][e]);
                    x[u] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, x[u]))));
                }
            }
            bool seen[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                seen[u] = row < rows && row_sees(a, g.span, own, v0 + sub + kLanes * u);
                x[u] = seen[u] ? x[u] * a.scale_log2 : -INFINITY;
            }
            float top = fmaxf(x[0], x[1]);
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top), base = mn == -INFINITY ? 0.f : mn;
            const float keep = exp2f(m - base);  // 0 while m = -inf
            float part = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float e = seen[u] ? exp2f(x[u] - base) : 0.f;
                s.p[row][sub + kLanes * u] = seen[u] ? e : -1.f;  // no weight is negative
                part += e;
            }
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
            l = l * keep + part;
            m = mn;
#pragma unroll
            for (int u = 0; u < NO; ++u) o[u] *= keep;
            __syncwarp();  // the row's weights come from threads of this warp only
#pragma unroll 8
            for (int kj = 0; kj < kKeys; ++kj) {
                const float p = s.p[row][kj];
                const bool adds = !(p < 0.f);  // a hidden place adds nothing, whatever v holds there
#pragma unroll
                for (int u = 0; u < NO; u += NC) {
                    const float *v = &s.v[kj][NC * sub + kLanes * u];
                    float y[NC];
                    if constexpr (NC == 4)
                        *reinterpret_cast<float4 *>(y) = *reinterpret_cast<const float4 *>(v);
                    else
                        *reinterpret_cast<float2 *>(y) = *reinterpret_cast<const float2 *>(v);
#pragma unroll
                    for (int e = 0; e < NC; ++e) o[u + e] = adds ? fmaf(p, y[e], o[u + e]) : o[u + e];
                }
            }
            __syncwarp();
        }
        const bool whole = g.i0 == 0 && g.i1 == g.span.n;
        if (row < rows) {
            const long long at = (long long)(g.req.row0 + tok) * a.Hq + g.h * a.G +
                                 (g.qt * kRows + row - tok * a.G);
            const float inv = whole ? 1.f / l : 1.f;
            float *part = a.part + (long long)part_slot(c, g) * kRows * (HD + 2);
#pragma unroll
            for (int u = 0; u < NO; u += NC) {
                const int col = NC * sub + kLanes * u;
                float *dst = whole ? static_cast<float *>(a.o) + at * HD + col
                                   : part + part_at<kRows>(row, col);
                if constexpr (NC == 4)
                    put(dst, make_float4(o[u] * inv, o[u + 1] * inv, o[u + 2] * inv, o[u + 3] * inv));
                else
                    *reinterpret_cast<float2 *>(dst) = make_float2(o[u] * inv, o[u + 1] * inv);
            }
            if (sub == 0) {
                if (!whole) {
                    part[kRows * HD + row] = m;
                    part[kRows * HD + kRows + row] = l;
                } else if (a.lse) {
                    a.lse[at] = (m + log2f(l)) * 0.69314718055994531f;
                }
            }
        }
        if (a.count && !whole)
            join_if_last<float, kRows, HD, kThreads>(a, c, g, cur.x, cur.N, cur.P, &s.join);
    }
    if (tid == 0 && !a.count) write_desc(a, c, g, any, cur.x, cur.N, cur.P);
}

// Joins the partials of the units that several workers hold: block (u, y) the rows y * RB
// on of the u-th of them.  A thread takes PER column groups (of four) of a row, CL apart, four
// partials at a time; the rows of a group lie side by side, so a warp reads whole lines.
// SLICES threads share a value's partials, added in the order of the workers and then of
// the slices.  The calls that come here have few units and many partials to each: small
// row blocks spread them over the SMs (16 drafts over 131072 places, 38 partials of
// 128 rows for each of eight units: 65.9 us a call with 32 rows a block, 62.5 with 16, 60.9 with 8).
template <int ROWS, int HD>
struct Combine {
    static constexpr int kThreads = 512;
    static constexpr int RB = 8;
    static constexpr int CL = HD == 256 ? 16 : 8;
    static constexpr int PER = HD / 4 / CL;
    static constexpr int SLICES = kThreads / (RB * CL);
};

template <typename T, int ROWS, int HD>
__global__ void __launch_bounds__(512) combine_kernel(const __grid_constant__ AttnArgs a, int workers) {
    using C = Combine<ROWS, HD>;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ __align__(16) unsigned char raw[sizeof(Partial<C::PER>) * (C::SLICES - 1) * C::RB * C::CL];
    Partial<C::PER>(*part)[C::RB * C::CL] = reinterpret_cast<Partial<C::PER>(*)[C::RB * C::CL]>(raw);
    // The unit of this block: the blockIdx.x-th worker that a unit to join begins in.
    __shared__ int found[C::kThreads / 32], unit;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const bool begins = (int)threadIdx.x < workers && a.desc[2 * threadIdx.x].x >= 0;
    const unsigned ballot = __ballot_sync(0xffffffffu, begins);
    if (lane == 0) found[warp] = __popc(ballot);
    if (threadIdx.x == 0) unit = -1;
    __syncthreads();
    int rank = __popc(ballot & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) rank += found[w];
    if (begins && rank == (int)blockIdx.x) unit = threadIdx.x;
    __syncthreads();
    const int c = unit;
    if (c < 0) return;
    const int4 d0 = a.desc[2 * c], d1 = a.desc[2 * c + 1];
    const int last = d0.x, qt = d0.y, h = d0.z, row0 = d0.w, T_r = d1.x, rb = blockIdx.y * C::RB;
    if (qt * ROWS + rb >= T_r * a.G) return;
    const int item = threadIdx.x % (C::RB * C::CL), slice = threadIdx.x / (C::RB * C::CL);
    const int row = rb + item % C::RB, cg = item / C::RB, i = qt * ROWS + row;
    Partial<C::PER> s;
    add_partials<ROWS, HD, C::PER, C::CL>(a, s, c, c + slice, C::SLICES, last, row, cg);
    if (slice > 0) part[slice - 1][item] = s;
    __syncthreads();
    if (slice > 0 || i >= T_r * a.G) return;
#pragma unroll 1
    for (int k = 0; k < C::SLICES - 1; ++k) s.add(part[k][item].m, part[k][item].l, part[k][item].o);
    const int t = div_group(a, i);
    const long long at = (long long)(row0 + t) * a.Hq + h * a.G + (i - t * a.G);
    const float inv = 1.f / s.l;
#pragma unroll
    for (int e = 0; e < C::PER; ++e)
        put(static_cast<T *>(a.o) + at * HD + 4 * (cg + e * C::CL),
            make_float4(s.o[e].x * inv, s.o[e].y * inv, s.o[e].z * inv, s.o[e].w * inv));
    if (a.lse && cg == 0) a.lse[at] = (s.m + log2f(s.l)) * 0.69314718055994531f;
}

template <typename K, typename... More>
cudaError_t launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   const AttnArgs &a, More... more) {
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
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

template <int HD>
cudaError_t launch_simple(const AttnArgs &a, cudaStream_t stream) {
    const cudaError_t e = allow_smem<attn_simple_kernel<HD>>((int)sizeof(Smem<HD>));
    if (e != cudaSuccess) return e;
    return launch(attn_simple_kernel<HD>, dim3(kAttnWorkers), kThreads, sizeof(Smem<HD>),
                  stream, a);
}

template <typename T, int ROWS, int HD>
cudaError_t launch_combine(const AttnArgs &a, int workers, cudaStream_t stream) {
    using C = Combine<ROWS, HD>;
    const long long units = (long long)a.B * a.Hkv * (((long long)a.max_T * a.G + ROWS - 1) / ROWS);
    if (units == 0) return cudaSuccess;  // max_T = 0: the rows are no request's
    return launch(combine_kernel<T, ROWS, HD>, dim3((unsigned)std::min<long long>(units, workers), ROWS / C::RB),
                  C::kThreads, 0, stream, a, workers);
}

// The launches of a call: finished units and partials, then the join where the first
// kernel does not do it.
template <int HD>
cudaError_t launch_hd(const AttnArgs &a, AttnKind kind, cudaStream_t stream) {
    if constexpr (HD == 64 || HD == 128) {
        if (kind == kAttnDrafts || kind == kAttnWide) {
            const cudaError_t e = launch_attn_tc(a, kind == kAttnWide, stream);
            if (e != cudaSuccess || a.count) return e;
            return kind == kAttnWide ? launch_combine<__nv_bfloat16, 256, HD>(a, kAttnTcWorkers, stream)
                                     : launch_combine<__nv_bfloat16, 128, HD>(a, kAttnWorkers, stream);
        }
    }
    const cudaError_t e = kind == kAttnSimple ? launch_simple<HD>(a, stream) : launch_attn_rows(a, stream);
    if (e != cudaSuccess || a.count) return e;
    return kind == kAttnSimple ? launch_combine<float, 16, HD>(a, kAttnWorkers, stream)
                               : launch_combine<__nv_bfloat16, 16, HD>(a, kAttnWorkers, stream);
}

}  // namespace

cudaError_t launch_attn(AttnArgs a, bool bf16, cudaStream_t stream) {
    // Few partials to a unit: the block that writes the last one joins them, and the second
    // launch is saved.  A request's key heads have equal work, so a unit spans at most
    // workers / key heads (and a bit) of them, and no more than its tiles allow.  On the tensor
    // cores a unit has many rows and a join is longer, so fewer partials are few; but with
    // units enough to keep every fourth worker busy most units lie in one or two workers, whatever
    // the bound says (64 requests' 16 drafts: 127.5 us joined by a launch, 124.5 so; 128 requests
    // behind a window: 75 and 72).  Those that do not, of a long request among short ones, are
    // joined group by group (16 drafts over 130000 places beside 39 requests of up to 90: 73 us;
    // all partials by the last warpgroup 226, by a launch 64).
    const AttnKind kind = attn_kind(bf16, a.hd, (long long)a.max_T * a.G);
    const bool tc = kind == kAttnDrafts || kind == kAttnWide;
    const int workers = kind == kAttnWide ? kAttnTcWorkers : kAttnWorkers;
    const int unit = kind == kAttnWide ? 256 : kind == kAttnDrafts ? 128 : 16;
    const long long tiles = ((long long)a.max_pages << a.page_shift) / (tc ? 64 : 32);
    const long long parts = std::min<long long>(workers / a.Hkv, tiles / 2) + 2;
    const long long units = (long long)a.B * a.Hkv * (((long long)a.max_T * a.G + unit - 1) / unit);
    if (parts > (tc ? 8 : kMaxParts) && !(tc && units * 4 >= workers)) a.count = nullptr;
    switch (a.hd) {
        case 32: return launch_hd<32>(a, kind, stream);
        case 64: return launch_hd<64>(a, kind, stream);
        case 128: return launch_hd<128>(a, kind, stream);
        default: return launch_hd<256>(a, kind, stream);
    }
}

// Which kernel runs, by type and rows a key head: float32 on the CUDA cores; up to
// 16 rows as one mma.sync tile; more on tcgen05, in units of 128 or 256 rows, for heads of
// 64 and 128 (those of 32 and 256 have the 16-row kernel only).  Prompt chunks in units of 128 rows would read the cache twice
// as often, and lose the second warpgroup that keeps the tensor cores busy: 4001 rows over
// 6007 places 704 us in units of 256 and 880 of 128, 8000 rows behind a window of 512
// 167 and 237.  Drafts in units of 256 rows, one block an SM: 64 requests' 16 drafts 137 us
// against 127.
AttnKind attn_kind(bool bf16, int hd, long long rows) {
    if (!bf16) return kAttnSimple;
    if (rows <= 16 || (hd != 64 && hd != 128)) return kAttnRows;
    return rows <= 128 ? kAttnDrafts : kAttnWide;
}

int64_t attn_workspace(bool bf16, int hd, long long rows) {
    const AttnKind kind = attn_kind(bf16, hd, rows);
    const int64_t workers = kind == kAttnWide ? kAttnTcWorkers : kAttnWorkers;
    const int64_t unit = kind == kAttnWide ? 256 : kind == kAttnDrafts ? 128 : 16;
    return kAttnHeader +
           2 * workers * unit * (hd + 2) * (int64_t)sizeof(float);
}

}  // namespace gdn
