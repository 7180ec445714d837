// Linear attention of drafts on the tensor cores (mma.sync): outputs only, bf16, dk 64 or 128, dv a
// multiple of 64, fewer rows than the prompts' kernel takes.
//
// The state before the drafts stays as it is, so all of a request's rows read the same one:
//     o_i = scale (d(i, -1) S^T q_i + sum_{j <= i} d(i, j) (q_i . k_j) v_j)
// Bound by the states' bytes (64 KB a head of 128 x 128).  A block holds dk x 64 of a state in
// registers as B operands: thread (g, c) of a warp holds rows 2c, 2c + 1,
// 2c + 8, 2c + 9 of a step's 16 and four columns from 4g, of which each belongs to another product
// of 8 columns.  An element is the sum of two bf16 terms, 2^-17 of itself off, and products are
// added up in float32; q and k are bf16 already.  A product has 16 rows of a draft, so few rows cost
// as much as 16.  All that takes as long as the loads, one block at a time, so a block goes on to
// further units: one thread asks the TMA engine for the next one's state and rows (128-byte swizzle)
// as soon as its own state is in registers.  Three blocks an SM, 42 KB of loads each in flight.
#include <cstdint>

#include "gdn_launch.h"
#include "gdn_linear.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = 4;  // that share a state's rows; two of each, by columns
constexpr int CV = 64;  // value columns of a block

__device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NG groups of 16 rows.
template <int DK, int NG>
struct Tiles {
    static constexpr int T = 16 * NG;
    static constexpr int BUFFERS = NG == 1 ? 2 : 1;  // of rows
    struct Rows {
        __nv_bfloat16 q[DK / 64][T][64], k[DK / 64][T][64], v[T][64];
    };
    float state[2][DK][32];
    Rows rows[BUFFERS];
    float red[kWarps][16][CV];  // (16 bytes c of a row lie at c ^ (row & 1): different banks)
    float d[T][T + 2];  // d[i][j + 1] = d(i, j)
    float g[T];
    unsigned long long full;  // barrier: a unit's state and rows are there
};

struct Launch {
    LinearArgs a;
    CUtensorMap q, k, v, pool;
    unsigned units;
};

__device__ __forceinline__ void tma(void *to, const CUtensorMap *map, int x, int y, uint32_t b) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(smem_addr(to)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(b)
        : "memory");
}

template <int DK, int NG>
__global__ void __launch_bounds__(kThreads, 3) drafts_kernel(const __grid_constant__ Launch L) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int KS = DK / 64;  // steps of 16 rows of the state a warp
    extern __shared__ __align__(1024) unsigned char raw[];
    Tiles<DK, NG> &s = *reinterpret_cast<Tiles<DK, NG> *>(raw);
    const LinearArgs &a = L.a;
    const gdn_linear &g = a.g;
    const unsigned units = L.units;
    const int tid = threadIdx.x, lane = tid & 31, gr = lane >> 2, c = lane & 3;
    const int warp = (tid >> 5) % kWarps, side = (tid >> 5) / kWarps;  // rows, and 32 columns
    const unsigned slices = g.dv / CV;
    const int kb = warp * (DK / kWarps);
    if (tid == 0) {
        mbar_init(bar(s.full), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();

    // A unit: rows (none: skip it), head, first value column, this thread's logarithm.
    struct Work {
        LinearUnit u;
        int h, c0;
        int row;  // the state's first row in the pool
        float g;
    };
    // Units in order, `step` at a time; a unit's words are loaded a round before they are looked at.
    struct Place {
        unsigned r, h, s;
    };
    auto place_of = [&](unsigned at) {
        const unsigned unit = at / slices;
        return Place{unit / (unsigned)g.heads, unit % (unsigned)g.heads, at - unit * slices};
    };
    struct Words {
        int c0, c1, slot;
        Place p;
    };
    auto words_of = [&](const Place &p) {
        Words x = {0, 0, -1, p};
        if (p.r >= (unsigned)g.batch) return x;
        x.slot = ld_early(g.slot_ids + p.r);
        if (g.cu_seqlens) {
            x.c0 = ld_early(g.cu_seqlens + p.r);
            x.c1 = ld_early(g.cu_seqlens + p.r + 1);
        } else {
            x.c0 = p.r * g.max_T;
            x.c1 = x.c0 + g.max_T;
        }
        return x;
    };
    auto work_of = [&](const Words &x) {
        Work w;
        w.u.T = w.u.row0 = 0;
        w.row = (x.slot * g.heads + (int)x.p.h) * DK;  // below 2^31: checked on the host
        w.h = x.p.h;
        w.c0 = x.p.s * CV;
        w.g = 0.f;
        if (x.p.r >= (unsigned)g.batch) return w;
        if (linear_words(a, x.c0, x.c1, x.slot, w.h, w.u) && tid < w.u.T)
            w.g = ld_early(g.log_decay + (long long)(w.u.row0 + tid) * g.decay_stride + w.h);
        return w;
    };
    // One thread's: the state and the rows of a unit.
    constexpr uint32_t kStateBytes = DK * CV * 4, kRowBytes = Tiles<DK, NG>::T * (2 * DK + CV) * 2;
    auto copy_state = [&](const Work &w) {
        for (int x = 0; x < 2; ++x) tma(s.state[x], &L.pool, w.c0 + 32 * x, w.row, bar(s.full));
    };
    auto copy_rows = [&](const Work &w, typename Tiles<DK, NG>::Rows &to) {
        const int col = w.h / a.group * DK;
        for (int x = 0; x < DK / 64; ++x) {
            tma(to.q[x], &L.q, col + 64 * x, w.u.row0, bar(s.full));
            tma(to.k[x], &L.k, col + 64 * x, w.u.row0, bar(s.full));
        }
        tma(to.v, &L.v, w.h * g.dv + w.c0, w.u.row0, bar(s.full));
    };
    // Bytes of a row of 64 columns of bf16: 16 bytes c lie at c ^ (row & 7).
    auto word = [](const __nv_bfloat16 (*tile)[64], int row, int col) {
        return *reinterpret_cast<const uint32_t *>(&tile[row][(col & 7) + 8 * ((col >> 3) ^ (row & 7))]);
    };

    constexpr bool AHEAD = Tiles<DK, NG>::BUFFERS == 2;
    const unsigned step = gridDim.x;  // (units and three steps fit 2^31)
    const Place by = place_of(step);
    auto advance = [&](Place &p) {
        p.s += by.s;
        p.h += by.h;
        p.r += by.r;
        if (p.s >= slices) {
            p.s -= slices;
            ++p.h;
        }
        if (p.h >= (unsigned)g.heads) {
            p.h -= g.heads;
            ++p.r;
        }
    };
    Place ahead = place_of(blockIdx.x);
    const Words first = words_of(ahead);
    advance(ahead);
    const Words second = words_of(ahead);
    Work w = work_of(first), next = work_of(second);
    int buffer = 0;
    uint32_t round = 0;
    auto ask = [&](const Work &x) {
        if (x.u.T > 0) arrive_expect(bar(s.full), kStateBytes + kRowBytes);
    };
    if (tid == 0 && w.u.T > 0) {
        ask(w);
        copy_state(w);
        copy_rows(w, s.rows[0]);
    }
    for (unsigned at = blockIdx.x; at < units; at += step) {
        const int T = w.u.T;
        typename Tiles<DK, NG>::Rows &rows_ = s.rows[buffer];
        advance(ahead);
        const Words coming = words_of(ahead);
        if (tid < T) s.g[tid] = w.g;
        if (T > 0) {
            const bool there = wait_parity(bar(s.full), round++ & 1);
            if (!__syncthreads_and(there)) {  // the copies never came: nothing more can be right
                if (tid == 0 && g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_TIMEOUT);
                return;
            }
        }
        // The state as operands: rows 2c, 2c + 1 (and 8 further), four columns from 4 gr.
        uint32_t hi[KS][4][2], lo[KS][4][2];
        if (T > 0) {
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const int row = kb + 16 * st + 8 * p + 2 * c;  // 16 bytes gr of it, and of the next
                    const float4 y = *reinterpret_cast<const float4 *>(&s.state[side][row][4 * (gr ^ (2 * c))]);
                    const float4 z =
                        *reinterpret_cast<const float4 *>(&s.state[side][row + 1][4 * (gr ^ (2 * c + 1))]);
                    const float y4[4] = {y.x, y.y, y.z, y.w}, z4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t b = pack(y4[t], z4[t]);
                        hi[st][t][p] = b;
                        lo[st][t][p] = pack(y4[t] - low(b), z4[t] - high(b));
                    }
                }
        }
        __syncthreads();
        if (tid == 0 && next.u.T > 0) {
            ask(next);
            copy_state(next);
            if (AHEAD) copy_rows(next, s.rows[buffer ^ 1]);
        }
        __syncwarp();
        // Row i's decays: sums from its end on, a lane a column (two where there are more rows).
        for (int i = tid >> 5; i < T; i += kThreads / 32) {
#pragma unroll
            for (int y = 0; y < (NG > 1 ? 2 : 1); ++y) {
                float sum = 0.f;  // of the logarithms of rows j + 1 to i
                const int j = 32 * y + lane - 1;
                if (NG == 1) {
                    sum = lane <= i ? s.g[lane] : 0.f;
#pragma unroll
                    for (int d = 1; d < 16; d <<= 1) {
                        const float z = __shfl_down_sync(0xffffffffu, sum, d);
                        if (lane + d <= i) sum += z;
                    }
                } else if (j < i) {
                    for (int l = j + 1; l <= i; ++l) sum += s.g[l];
                }
                if (j <= i) s.d[i][j + 1] = j == i ? 1.f : expf(sum);
            }
        }

        __syncthreads();
#pragma unroll 1
        for (int m = 0; 16 * m < T; ++m) {
            uint32_t A[KS][4];
            float acc[4][4] = {};
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                        A[st][x] = word(rows_.q[(kb + 16 * st) / 64], 16 * m + gr + 8 * (x & 1),
                                    (kb + 16 * st) % 64 + 8 * (x >> 1) + 2 * c);
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int t = 0; t < 4; ++t) mma(acc[t], A[st], lo[st][t][0], lo[st][t][1]);
#pragma unroll
            for (int st = 0; st < KS; ++st)
#pragma unroll
                for (int t = 0; t < 4; ++t) mma(acc[t], A[st], hi[st][t][0], hi[st][t][1]);
            // Rows gr and gr + 8 of the group.
            const int i0 = 16 * m + gr, i1 = i0 + 8;
            const float from0 = i0 < T ? s.d[i0][0] : 0.f, from1 = i1 < T ? s.d[i1][0] : 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                acc[t][0] *= from0;
                acc[t][1] *= from0;
                acc[t][2] *= from1;
                acc[t][3] *= from1;
            }
            // The rows' own products, this warp's share of dk: with their decays they are the weights of
            // the values, as operands of the next product just where they are.
            for (int l = 0; l <= m; ++l) {
                uint32_t W[4], R[4];  // two terms
                const auto weights = [&](int n) {
                    float own[4] = {};
#pragma unroll
                    for (int st = 0; st < KS; ++st) {
                        const auto *key = rows_.k[(kb + 16 * st) / 64];
                        const int j = 16 * l + 8 * n + gr, col = (kb + 16 * st) % 64 + 2 * c;
                        mma(own, A[st], word(key, j, col), word(key, j, col + 8));
                    }
                    const int j = 16 * l + 8 * n + 2 * c;
                    const float w0 = j <= i0 && i0 < T ? own[0] * s.d[i0][j + 1] : 0.f;
                    const float w1 = j < i0 && i0 < T ? own[1] * s.d[i0][j + 2] : 0.f;
                    const float w2 = j <= i1 && i1 < T ? own[2] * s.d[i1][j + 1] : 0.f;
                    const float w3 = j < i1 && i1 < T ? own[3] * s.d[i1][j + 2] : 0.f;
                    W[2 * n] = pack(w0, w1);
                    W[2 * n + 1] = pack(w2, w3);
                    R[2 * n] = pack(w0 - low(W[2 * n]), w1 - high(W[2 * n]));
                    R[2 * n + 1] = pack(w2 - low(W[2 * n + 1]), w3 - high(W[2 * n + 1]));
                };
                weights(0);
                weights(1);
                // Four columns of values from 4 gr, of rows 2c, 2c + 1 and 8 further (0 where there are none:
                // their weights are 0, and they hold whatever lay there).
                uint2 v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int j = 16 * l + 2 * c + (x & 1) + 8 * (x >> 1), col = 32 * side + 4 * gr;
                    v[x] = j < T ? *reinterpret_cast<const uint2 *>(
                                       &rows_.v[j][(col & 7) + 8 * ((col >> 3) ^ (j & 7))])
                                 : make_uint2(0u, 0u);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t take = t & 1 ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(t < 2 ? v[0].x : v[0].y, t < 2 ? v[1].x : v[1].y, take);
                    const uint32_t b1 = __byte_perm(t < 2 ? v[2].x : v[2].y, t < 2 ? v[3].x : v[3].y, take);
                    mma(acc[t], R, b0, b1);
                    mma(acc[t], W, b0, b1);
                }
            }
            // Column 2c (2c + 1) of product t is column 8c (+ 4) + t of the warp's 32.
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    *reinterpret_cast<float4 *>(
                        &s.red[warp][gr + 8 * i][4 * ((8 * side + 2 * c + n) ^ (gr & 1))]) =
                        make_float4(acc[0][2 * i + n], acc[1][2 * i + n], acc[2][2 * i + n], acc[3][2 * i + n]);
            __syncthreads();
            const int rows = min(16, T - 16 * m);
            for (int e = tid; e < rows * (CV / 4); e += kThreads) {
                const int i = e / (CV / 4), col = e % (CV / 4) * 4, row = 16 * m + i;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float4 y = *reinterpret_cast<const float4 *>(&s.red[x][i][4 * ((col / 4) ^ (i & 1))]);
                    o.x += y.x;
                    o.y += y.y;
                    o.z += y.z;
                    o.w += y.w;
                }
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) +
                                           ((long long)(w.u.row0 + row) * g.heads + w.h) * g.dv + w.c0 + col) =
                    make_uint2(pack(o.x * g.scale, o.y * g.scale), pack(o.z * g.scale, o.w * g.scale));
            }
            __syncthreads();
        }
        if (AHEAD)
            buffer ^= 1;
        else
            if (tid == 0 && next.u.T > 0) copy_rows(next, s.rows[0]);  // all have left this unit's
        w = next;
        next = work_of(coming);
    }
}

bool encode(CUtensorMap *map, CUtensorMapDataType type, const void *base, long long cols, long long rows,
            long long stride, int esz, int box_cols, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(stride * esz)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    const cuuint32_t elem[2] = {1, 1};
    return encoder()(map, type, 2, const_cast<void *>(base), dims, strides, box, elem,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int NG>
cudaError_t launch_one(const LinearArgs &a, cudaStream_t stream) {
    const gdn_linear &g = a.g;
    constexpr int smem = (int)sizeof(Tiles<DK, NG>), T = Tiles<DK, NG>::T;
    Launch L;
    L.a = a;
    L.units = (unsigned)g.batch * g.heads * (g.dv / CV);  // at most 2^30
    const long long krow = (long long)g.k_heads * g.dk, vrow = (long long)g.heads * g.dv;
    if (!encoder() ||
        !encode(&L.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.q, krow, g.n_tok, g.q_stride, 2, 64, T) ||
        !encode(&L.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.k, krow, g.n_tok, g.k_stride, 2, 64, T) ||
        !encode(&L.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.v, vrow, g.n_tok, g.v_stride, 2, 64, T) ||
        !encode(&L.pool, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, g.pool, g.dv, g.pool_slots * g.heads * g.dk, g.dv, 4, 32,
                DK))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<drafts_kernel<DK, NG>>(smem);
    if (e != cudaSuccess) return e;
    constexpr int fit = 233472 / (smem + 1024), per_sm = fit < 3 ? fit : 3;
    static_assert(per_sm >= 1, "");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.units < 152 * per_sm ? L.units : 152 * per_sm);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, drafts_kernel<DK, NG>, L);
}

}  // namespace

bool linear_drafts_runs(const gdn_linear &g) {
    return g.dtype == GDN_BF16 && (g.dk == 64 || g.dk == 128) && g.dv % CV == 0 && g.max_T > 1 && g.max_T <= 48 &&
           g.pool_slots * g.heads * g.dk <= 0x7fffffffLL;  // the pool's rows are numbered in 32 bits
}

cudaError_t launch_linear_drafts(const LinearArgs &a, cudaStream_t stream) {
    if (a.g.dk == 64) return a.g.max_T <= 16 ? launch_one<64, 1>(a, stream) : launch_one<64, 3>(a, stream);
    return a.g.max_T <= 16 ? launch_one<128, 1>(a, stream) : launch_one<128, 3>(a, stream);
}

}  // namespace gdn
