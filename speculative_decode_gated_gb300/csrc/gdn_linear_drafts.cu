// Linear attention of drafts on the tensor cores (mma.sync): outputs only, bf16, dk 64 or 128, dv a
// multiple of 64, fewer rows than the prompts' kernel takes.
//
// The state before the drafts stays as it is, so all of a request's rows read the same one:
//     o_i = scale (d(i, -1) S^T q_i + sum_{j <= i} d(i, j) (q_i . k_j) v_j)
// Bound by the states' bytes (64 KB a head of 128 x 128).  A block holds dk x 64 of a state in
// registers, where the loads leave it as B operands: thread (g, c) of a warp holds rows 2c, 2c + 1,
// 2c + 8, 2c + 9 of a step's 16 and four columns from 4g, of which each belongs to another product
// of 8 columns.  An element is the sum of two bf16 terms, 2^-17 of itself off, and products are
// added up in float32; q and k are bf16 already.  A product has 16 rows of a draft, so few rows cost
// as much as 16: that, and the few tokens' own products, hides behind the state's stream.
#include <cstdint>

#include "gdn_launch.h"
#include "gdn_linear.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128, kWarps = 4;
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
__global__ void __launch_bounds__(kThreads, 4) drafts_kernel(const LinearArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int T = 16 * NG, KS = DK / 64;  // most rows; steps of 16 rows of the state a warp
    __shared__ __align__(16) __nv_bfloat16 sv[T][CV];
    __shared__ __align__(16) float red[kWarps][16][CV];
    __shared__ float part[kWarps][16][T + 1];
    __shared__ float sd[T][T + 2];  // sd[i][j + 1] = d(i, j)
    __shared__ float sg[T];
    const gdn_linear &g = a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, c = lane & 3;
    const int slices = g.dv / CV;
    const int unit = blockIdx.x / slices, c0 = (blockIdx.x - unit * slices) * CV;
    const int r = unit / g.heads, h = unit - r * g.heads;
    LinearUnit u;
    if (!linear_unit(a, r, h, false, u)) return;

    // The state.
    const int kb = warp * (DK / kWarps);
    float4 S[KS][4][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float *row = u.tile + (long long)(kb + 16 * s + 2 * c + (i & 1) + 8 * (i >> 1)) * g.dv + c0 + 4 * gr;
#pragma unroll
            for (int x = 0; x < 2; ++x) S[s][i][x] = __ldcs(reinterpret_cast<const float4 *>(row + 32 * x));
        }

    // The rows: values and logarithms to shared memory, queries and keys as operands.
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(g.q) + (long long)(h / a.group) * DK + kb + 2 * c;
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(g.k) + (long long)(h / a.group) * DK + kb + 2 * c;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(g.v) + (long long)h * g.dv + c0;
    auto word = [&](const __nv_bfloat16 *x, long long stride, int i, int off) {
        return i < u.T ? __ldg(reinterpret_cast<const uint32_t *>(x + (u.row0 + i) * stride + off)) : 0u;
    };
    for (int e = tid; e < u.T * (CV / 8); e += kThreads) {
        const int i = e / (CV / 8), x = e % (CV / 8) * 8;
        *reinterpret_cast<uint4 *>(&sv[i][x]) =
            __ldg(reinterpret_cast<const uint4 *>(v + (u.row0 + i) * g.v_stride + x));
    }
    if (tid < u.T) sg[tid] = __ldg(g.log_decay + (long long)(u.row0 + tid) * g.decay_stride + h);
    __syncthreads();
    // Column j + 1 of the decays: sums down the column.
    if (tid <= u.T) {
        float sum = 0.f;
        if (tid > 0) sd[tid - 1][tid] = 1.f;
        for (int i = tid; i < u.T; ++i) {
            sum += sg[i];
            sd[i][tid] = expf(sum);
        }
    }

    uint32_t hi[KS][8][2], lo[KS][8][2];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float4 y = S[s][2 * p][x], z = S[s][2 * p + 1][x];
                const float y4[4] = {y.x, y.y, y.z, y.w}, z4[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t w = pack(y4[t], z4[t]);
                    hi[s][4 * x + t][p] = w;
                    lo[s][4 * x + t][p] = pack(y4[t] - low(w), z4[t] - high(w));
                }
            }

#pragma unroll 1
    for (int m = 0; 16 * m < u.T; ++m) {
        uint32_t A[KS][4];
        float acc[8][4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                A[s][x] = word(q, g.q_stride, 16 * m + gr + 8 * (x & 1), 16 * s + 8 * (x >> 1));
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                mma(acc[t], A[s], lo[s][t][0], lo[s][t][1]);
                mma(acc[t], A[s], hi[s][t][0], hi[s][t][1]);
            }
        // Column 2c (2c + 1) of product t is column 32 (t / 4) + 8c (+ 4) + t % 4.
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    *reinterpret_cast<float4 *>(&red[warp][gr + 8 * i][32 * x + 8 * c + 4 * n]) =
                        make_float4(acc[4 * x][2 * i + n], acc[4 * x + 1][2 * i + n], acc[4 * x + 2][2 * i + n],
                                    acc[4 * x + 3][2 * i + n]);
        // The rows' own products.
        for (int l = 0; l <= m; ++l) {
            float own[2][4] = {};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    mma(own[n], A[s], word(k, g.k_stride, 16 * l + 8 * n + gr, 16 * s),
                        word(k, g.k_stride, 16 * l + 8 * n + gr, 16 * s + 8));
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    part[warp][gr + 8 * (x >> 1)][16 * l + 8 * n + 2 * c + (x & 1)] = own[n][x];
        }
        __syncthreads();
        // With their decays, over the first warp's share.
        const int rows = min(16, u.T - 16 * m);
        for (int e = tid; e < 16 * 16 * (m + 1); e += kThreads) {
            const int i = e & 15, j = e >> 4, row = 16 * m + i;
            if (i < rows && j <= row)
                part[0][i][j] = ((part[0][i][j] + part[1][i][j]) + (part[2][i][j] + part[3][i][j])) * sd[row][j + 1];
        }
        __syncthreads();
        for (int e = tid; e < rows * (CV / 4); e += kThreads) {
            const int i = e / (CV / 4), col = e % (CV / 4) * 4, row = 16 * m + i;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(&red[w][i][col]);
                s.x += y.x;
                s.y += y.y;
                s.z += y.z;
                s.w += y.w;
            }
            const float d = sd[row][0];
            s = make_float4(s.x * d, s.y * d, s.z * d, s.w * d);
            for (int j = 0; j <= row; ++j) {
                const float x = part[0][i][j];
                const uint2 y = *reinterpret_cast<const uint2 *>(&sv[j][col]);
                s.x = fmaf(x, low(y.x), s.x);
                s.y = fmaf(x, high(y.x), s.y);
                s.z = fmaf(x, low(y.y), s.z);
                s.w = fmaf(x, high(y.y), s.w);
            }
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) +
                                       ((long long)(u.row0 + row) * g.heads + h) * g.dv + c0 + col) =
                make_uint2(pack(s.x * g.scale, s.y * g.scale), pack(s.z * g.scale, s.w * g.scale));
        }
        if (16 * (m + 1) < u.T) __syncthreads();
    }
}

template <int DK, int NG>
cudaError_t launch_one(const LinearArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.g.batch * a.g.heads * (a.g.dv / CV)));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, drafts_kernel<DK, NG>, a);
}

}  // namespace

bool linear_drafts_runs(const gdn_linear &g) {
    return g.dtype == GDN_BF16 && (g.dk == 64 || g.dk == 128) && g.dv % CV == 0 && g.max_T > 1 && g.max_T <= 48;
}

cudaError_t launch_linear_drafts(const LinearArgs &a, cudaStream_t stream) {
    if (a.g.dk == 64) return a.g.max_T <= 16 ? launch_one<64, 1>(a, stream) : launch_one<64, 3>(a, stream);
    return a.g.max_T <= 16 ? launch_one<128, 1>(a, stream) : launch_one<128, 3>(a, stream);
}

}  // namespace gdn
