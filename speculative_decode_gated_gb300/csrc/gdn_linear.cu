// Linear attention with a decay for each head, on CUDA cores: single tokens, drafts and their
// commits, float32, and every head size.
//
// With S the state before a block of up to C rows, d(i, j) = e^{g_{j+1} + ... + g_i} the decay
// from row j to row i (d(i, -1): from before the block),
//     o_i = scale (d(i, -1) S^T q_i + sum_{j <= i} d(i, j) (q_i . k_j) v_j)
//     S  <- d(n - 1, -1) S + sum_j d(n - 1, j) k_j v_j^T
// which needs one multiply-add a state element and row for each of the two, where the recurrence
// row by row needs two for the second.  Each decay is the exponential of a sum (products of
// rounded decays would be off by as many roundings as rows), and each sum is its own, so nothing
// cancels and a decay of 0 (g = -infinity) is no special case.
//
// A block holds dk x CV of a state in registers, a thread R rows of four columns, two rows to a
// packed float32 operand.  Blocks of later rows follow with the state in place.
// Bound by the state's bytes up to 16 or so rows: 64 KB a head of 128 x 128, read, and written
// too by a step or a commit.  64 single tokens of 32 such heads take 42 us (95% of the copy's rate),
// a commit of up to 16 rows of each of these requests 39 us (86%), one token 4 us, a launch.
#include <cstdint>

#include "gdn_launch.h"
#include "gdn_linear.cuh"

namespace gdn {
namespace {

template <typename T, int DK_, int CV_, int C_>
struct Shape {
    static constexpr int DK = DK_, CV = CV_, C = C_;
    static constexpr int CG = CV / 4;                                     // column groups
    static constexpr int NT = DK * CV / 64 > 128 ? DK * CV / 64 : 128;   // threads
    static constexpr int RG = NT / CG, R = DK / RG;                       // row groups, rows of each
    static constexpr int NW = NT / 32;
    static constexpr int KS = DK + 4;                                     // row stride of keys in shared memory
    static_assert(R >= 2 && R % 2 == 0 && R <= 16, "");
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
        " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// 16 bytes of a row as float32 to shared memory.
__device__ __forceinline__ void stage(float *dst, const float *src) {
    *reinterpret_cast<float4 *>(dst) = __ldg(reinterpret_cast<const float4 *>(src));
}
__device__ __forceinline__ void stage(float *dst, const __nv_bfloat16 *src) {
    float x[8];
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4 *>(src)), x);
    *reinterpret_cast<float4 *>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void put4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 x) {  // rounded once, to nearest even
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                                               *reinterpret_cast<const uint32_t *>(&hi));
}

template <typename T, int DK, int CV, int C, int MODE>
__global__ void __launch_bounds__(Shape<T, DK, CV, C>::NT) linear_kernel(const LinearArgs a) {
    using P = Shape<T, DK, CV, C>;
    constexpr int CG = P::CG, NT = P::NT, R = P::R, NW = P::NW, KS = P::KS, VE = 16 / (int)sizeof(T);
    constexpr bool OUT = MODE != kCommit, STATE = MODE != kVerify;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ __align__(16) float sq[OUT ? C : 1][KS], sk[C][KS], sv[C][CV];
    __shared__ __align__(16) float red[OUT ? NW : 1][C][CV];
    __shared__ float sd[C + 1][C + 1];  // sd[i][j + 1] = d(i, j)
    __shared__ float sa[C][C + 1];
    const gdn_linear &g = a.g;
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, lane = tid & 31, warp = tid >> 5;
    const int slices = g.dv / CV;
    const int unit = blockIdx.x / slices, c0 = (blockIdx.x - unit * slices) * CV;
    const int r = unit / g.heads, h = unit - r * g.heads;
    LinearUnit u;
    if (!linear_unit(a, r, h, MODE == kCommit, u)) return;

    // Element (rg R + i, c0 + 4 cg + c) of the state is S[i / 2][c].x or .y.
    float *tile = u.tile + (long long)(rg * R) * g.dv + c0 + 4 * cg;
    float2 S[R / 2][4];
#pragma unroll
    for (int i = 0; i < R / 2; ++i) {
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(tile + (long long)(2 * i) * g.dv));
        const float4 y = __ldcs(reinterpret_cast<const float4 *>(tile + (long long)(2 * i + 1) * g.dv));
        S[i][0] = make_float2(x.x, y.x);
        S[i][1] = make_float2(x.y, y.y);
        S[i][2] = make_float2(x.z, y.z);
        S[i][3] = make_float2(x.w, y.w);
    }
    const T *q = static_cast<const T *>(g.q) + (long long)(h / a.group) * DK;
    const T *k = static_cast<const T *>(g.k) + (long long)(h / a.group) * DK;
    const T *v = static_cast<const T *>(g.v) + (long long)h * g.dv + c0;
    T *o = static_cast<T *>(a.o);

#pragma unroll 1
    for (int t0 = 0; t0 < u.T; t0 += C) {
        const int n = min(C, u.T - t0);
        const long long row = u.row0 + t0;
        if (t0 > 0) __syncthreads();  // the last block of rows is done with
        for (int e = tid; e < n * (DK / VE); e += NT) {
            const int i = e / (DK / VE), c = e % (DK / VE) * VE;
            if (OUT) stage(&sq[i][c], q + (row + i) * g.q_stride + c);
            stage(&sk[i][c], k + (row + i) * g.k_stride + c);
        }
        for (int e = tid; e < n * (CV / VE); e += NT) {
            const int i = e / (CV / VE), c = e % (CV / VE) * VE;
            stage(&sv[i][c], v + (row + i) * g.v_stride + c);
        }
        // Column j + 1 of the decays: sums down the column.
        if (tid <= n) {
            float gs[C], sum = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i)
                gs[i] = i < n ? __ldg(g.log_decay + (row + i) * g.decay_stride + h) : 0.f;
            if (tid > 0) sd[tid - 1][tid] = 1.f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                sum += i >= tid ? gs[i] : 0.f;
                if (i >= tid && i < n) sd[i][tid] = expf(sum);
            }
        }
        __syncthreads();
        if (C == 1) {
            const float d = sd[0][0];
            const float4 v4 = *reinterpret_cast<const float4 *>(&sv[0][4 * cg]);
            const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
            float2 acc[4] = {};
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const float2 k2 = *reinterpret_cast<const float2 *>(&sk[0][rg * R + 2 * i]);
                float2 q2;
                if (OUT) q2 = *reinterpret_cast<const float2 *>(&sq[0][rg * R + 2 * i]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    S[i][c] = fma2(k2, make_float2(vv[c], vv[c]), mul2(S[i][c], make_float2(d, d)));
                    if (OUT) acc[c] = fma2(q2, S[i][c], acc[c]);
                }
            }
            if (OUT) {
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[c] = acc[c].x + acc[c].y;
#pragma unroll
                    for (int m = CG; m < 32; m <<= 1) x[c] += __shfl_xor_sync(0xffffffffu, x[c], m);
                }
                if (lane < CG) put4(&red[warp][0][4 * lane], make_float4(x[0], x[1], x[2], x[3]));
                __syncthreads();
                if (tid < CG) {
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float4 y = *reinterpret_cast<const float4 *>(&red[w][0][4 * tid]);
                        s.x += y.x;
                        s.y += y.y;
                        s.z += y.z;
                        s.w += y.w;
                    }
                    put4(o + (row * g.heads + h) * g.dv + c0 + 4 * tid,
                         make_float4(s.x * g.scale, s.y * g.scale, s.z * g.scale, s.w * g.scale));
                }
            }
            continue;
        }
        if (OUT) {
            // The rows' own products, with their decays.
            for (int e = tid; e < n * n; e += NT) {
                const int i = e / n, j = e - i * n;
                if (j > i) continue;
                float x = 0.f;
#pragma unroll 8
                for (int c = 0; c < DK; c += 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(&sq[i][c]);
                    const float4 z = *reinterpret_cast<const float4 *>(&sk[j][c]);
                    x = fmaf(y.x, z.x, fmaf(y.y, z.y, fmaf(y.z, z.z, fmaf(y.w, z.w, x))));
                }
                sa[i][j] = x * sd[i][j + 1];
            }
            // S^T q_i, a share of the rows a warp.
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                float2 acc[4] = {};
#pragma unroll
                for (int m = 0; m < R / 2; ++m) {
                    const float2 q2 = *reinterpret_cast<const float2 *>(&sq[i][rg * R + 2 * m]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[c] = fma2(q2, S[m][c], acc[c]);
                }
                float x[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[c] = acc[c].x + acc[c].y;
#pragma unroll
                    for (int m = CG; m < 32; m <<= 1) x[c] += __shfl_xor_sync(0xffffffffu, x[c], m);
                }
                if (lane < CG) put4(&red[warp][i][4 * lane], make_float4(x[0], x[1], x[2], x[3]));
            }
        }
        if (STATE || t0 + C < u.T) {
            const float keep = sd[n - 1][0];
#pragma unroll
            for (int i = 0; i < R / 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[i][c] = mul2(S[i][c], make_float2(keep, keep));
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const float d = sd[n - 1][j + 1];
                const float4 v4 = *reinterpret_cast<const float4 *>(&sv[j][4 * cg]);
                const float vv[4] = {v4.x * d, v4.y * d, v4.z * d, v4.w * d};
#pragma unroll
                for (int i = 0; i < R / 2; ++i) {
                    const float2 k2 = *reinterpret_cast<const float2 *>(&sk[j][rg * R + 2 * i]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) S[i][c] = fma2(k2, make_float2(vv[c], vv[c]), S[i][c]);
                }
            }
        }
        if (OUT) {
            __syncthreads();
            for (int e = tid; e < n * CG; e += NT) {
                const int i = e / CG, c = e % CG * 4;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float4 y = *reinterpret_cast<const float4 *>(&red[w][i][c]);
                    s.x += y.x;
                    s.y += y.y;
                    s.z += y.z;
                    s.w += y.w;
                }
                const float d = sd[i][0];
                s = make_float4(s.x * d, s.y * d, s.z * d, s.w * d);
                for (int j = 0; j <= i; ++j) {
                    const float x = sa[i][j];
                    const float4 y = *reinterpret_cast<const float4 *>(&sv[j][c]);
                    s.x = fmaf(x, y.x, s.x);
                    s.y = fmaf(x, y.y, s.y);
                    s.z = fmaf(x, y.z, s.z);
                    s.w = fmaf(x, y.w, s.w);
                }
                put4(o + ((row + i) * g.heads + h) * g.dv + c0 + c,
                     make_float4(s.x * g.scale, s.y * g.scale, s.z * g.scale, s.w * g.scale));
            }
        }
    }
    if (STATE) {
#pragma unroll
        for (int i = 0; i < R / 2; ++i) {
            __stcs(reinterpret_cast<float4 *>(tile + (long long)(2 * i) * g.dv),
                   make_float4(S[i][0].x, S[i][1].x, S[i][2].x, S[i][3].x));
            __stcs(reinterpret_cast<float4 *>(tile + (long long)(2 * i + 1) * g.dv),
                   make_float4(S[i][0].y, S[i][1].y, S[i][2].y, S[i][3].y));
        }
    }
}

template <typename T, int DK, int CV, int C, int MODE>
cudaError_t launch_one(const LinearArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.g.batch * a.g.heads * (a.g.dv / CV)));
    cfg.blockDim = dim3(Shape<T, DK, CV, C>::NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, linear_kernel<T, DK, CV, C, MODE>, a);
}

template <typename T, int DK, int CV, int C>
cudaError_t launch_mode(const LinearArgs &a, int mode, cudaStream_t stream) {
    switch (mode) {
        case kVerify: return launch_one<T, DK, CV, C, kVerify>(a, stream);
        case kCommit: return launch_one<T, DK, CV, C, kCommit>(a, stream);
        default: return launch_one<T, DK, CV, C, kFused>(a, stream);
    }
}

// Rows at a time: 16, or 8 where shared memory (48 KB) holds no more.
template <typename T, int DK, int CV>
cudaError_t launch_rows(const LinearArgs &a, int mode, cudaStream_t stream) {
    if (a.g.max_T == 1) return launch_mode<T, DK, CV, 1>(a, mode, stream);
    return launch_mode<T, DK, CV, DK == 256 ? 8 : 16>(a, mode, stream);
}

template <typename T, int DK>
cudaError_t launch_dk(const LinearArgs &a, int mode, cudaStream_t stream) {
    return a.g.dv % 64 == 0 ? launch_rows<T, DK, 64>(a, mode, stream) : launch_rows<T, DK, 32>(a, mode, stream);
}

template <typename T>
cudaError_t launch_type(const LinearArgs &a, int mode, cudaStream_t stream) {
    switch (a.g.dk) {
        case 32: return launch_dk<T, 32>(a, mode, stream);
        case 64: return launch_dk<T, 64>(a, mode, stream);
        case 128: return launch_dk<T, 128>(a, mode, stream);
        default: return launch_dk<T, 256>(a, mode, stream);
    }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int mode, cudaStream_t stream) {
    if (linear_tc_runs(a.g)) return launch_linear_tc(a, mode, stream);
    if (mode == kVerify && linear_drafts_runs(a.g)) return launch_linear_drafts(a, stream);
    return a.g.dtype == GDN_BF16 ? launch_type<__nv_bfloat16>(a, mode, stream)
                                 : launch_type<float>(a, mode, stream);
}

}  // namespace gdn
