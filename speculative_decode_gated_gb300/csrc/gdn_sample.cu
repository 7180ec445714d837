// Accepted lengths and next tokens of sampled drafts (gdn_accept_sample; the rule is
// in gdn.h).
//
// A draft stays if u q(x) < p(x): the product of two float32 is exact in float64.  The next
// token is found by its place in a running sum over a whole vocabulary, where a sum of float32
// (or one in another order) would move some border past the random number once in some
// thousand tokens.  So the weights are whole numbers, units of 2^-44: sums are exact in 64 bits
// (at most 2^18 of at most 2^44), and the token does not depend on how the row was divided.
//
// Bound by the bytes of one row of p, and one of q where a draft did not stay, a request.
// A cluster of CS blocks takes a request, each block a stretch of the row and each warp a
// stretch of that: first every warp's sum, then, by the sums of all warps, the one warp
// whose stretch holds the token reads it again (from L2) for the place.
#include <cstdint>

#include "gdn_device.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 512;  // ids that a warp takes at a time: four vectors a lane

using u64 = unsigned long long;

// Whole units of 2^-44; NaN and below 0: none, above 1: 2^44.
__device__ __forceinline__ u64 units(float x) {
    x = fminf(fmaxf(x, 0.f), 1.f);  // of NaN and 0 the maximum is 0
    return __float2ull_rz(x * 0x1p44f);  // an exact product
}

// The weights of one request's row.
struct Row {
    const float *p, *q;  // q = NULL: all of p, or of a lookup's draft
    int point;           // the id of a looked-up draft that did not stay (its weight is p - 1, so 0), or -1
    __device__ __forceinline__ u64 weight(int i, float x, float y) const {
        const u64 a = units(x);
        if (q) {
            const u64 b = units(y);
            return a > b ? a - b : 0;
        }
        return i == point ? 0 : a;
    }
};

__device__ __forceinline__ u64 warp_sum(u64 x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                     : "memory");
}
// Reads a 64-bit word of block `rank`'s shared memory.
__device__ __forceinline__ u64 peer_word(const u64 *mine, uint32_t rank) {
    uint32_t at = (uint32_t)__cvta_generic_to_shared(mine), there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
    u64 x;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(there) : "memory");
    return x;
}

struct Shared {
    u64 warp_total[kWarps];
    int accepted, from;  // rows kept; the row of p (and q) the next token comes from
    int point, rejected, ok;
};

// This lane's share of the sum of the weights of ids [i0, i1).
template <bool VEC>
__device__ __forceinline__ u64 lane_sum(const Row &w, int i0, int i1, int lane) {
    u64 sum = 0;
    if (VEC) {  // i0 is a multiple of 4, the rows are 16-byte aligned
        int i = i0 + lane * 4;
        for (; i + 384 + 3 < i1; i += kTile) {
            float4 x[4], y[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u] = __ldg(reinterpret_cast<const float4 *>(w.p + i + 128 * u));
                y[u] = w.q ? __ldg(reinterpret_cast<const float4 *>(w.q + i + 128 * u))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = i + 128 * u;
                sum += w.weight(j, x[u].x, y[u].x) + w.weight(j + 1, x[u].y, y[u].y) +
                       w.weight(j + 2, x[u].z, y[u].z) + w.weight(j + 3, x[u].w, y[u].w);
            }
        }
        for (; i < i1; i += 128)
            for (int e = 0; e < 4 && i + e < i1; ++e)
                sum += w.weight(i + e, w.p[i + e], w.q ? w.q[i + e] : 0.f);
        return sum;
    }
    int i = i0 + lane;
    for (; i + 7 * 32 < i1; i += 8 * 32) {
        float x[8], y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            x[u] = __ldg(w.p + i + 32 * u);
            y[u] = w.q ? __ldg(w.q + i + 32 * u) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += w.weight(i + 32 * u, x[u], y[u]);
    }
    for (; i < i1; i += 32) sum += w.weight(i, w.p[i], w.q ? w.q[i] : 0.f);
    return sum;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads)
    sample_kernel(const gdn_sample g, long long n_tok, int stretch, int32_t *accepted, int32_t *next_ids) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Shared s;
    uint32_t cs;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    const uint32_t rank = cluster_rank();
    const int r = blockIdx.x / cs;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // Which drafts stay: a lane a row, 32 rows at a time.  Every block finds out for itself.
    if (warp == 0) {
        long long c0 = (long long)r * g.max_T, c1 = c0 + g.max_T;
        if (g.cu_seqlens) {
            c0 = g.cu_seqlens[r];
            c1 = g.cu_seqlens[r + 1];
        }
        const bool ok = c1 >= c0 && c1 - c0 <= g.max_T && c0 >= 0 && c1 <= n_tok;
        const int T = ok ? (int)(c1 - c0) : 0;
        int a = T, point = -1;
        bool rejected = false;
        for (int t0 = 1; t0 < T; t0 += 32) {
            const int t = t0 + lane;
            bool stays = true;
            int x = 0;
            if (t < T) {
                x = g.draft_ids[c0 + t];
                stays = false;
                if (x >= 0 && x < g.vocab) {
                    const float p = g.target_probs[(c0 + t - 1) * g.target_stride + x];
                    const float q = g.draft_probs ? g.draft_probs[(c0 + t - 1) * g.draft_stride + x] : 1.f;
                    stays = (double)g.u_accept[c0 + t] * (double)q < (double)p;
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, !stays);
            if (m) {
                const int first = __ffs(m) - 1;
                a = t0 + first;
                point = __shfl_sync(0xffffffffu, x, first);
                rejected = true;
                if (lane == first && rank == 0 && g.dev_err && (x < 0 || x >= g.vocab))
                    atomicOr(g.dev_err, GDN_DEVERR_TOKEN);
                break;
            }
        }
        if (lane == 0) {
            s.ok = ok && T > 0;
            s.accepted = a;
            s.from = (int)(c0 + a - 1);
            s.rejected = rejected;
            s.point = point;
            if (rank == 0) {
                if (ok) accepted[r] = a;
                if (ok && T == 0) next_ids[r] = -1;
                if (!ok && g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_SEQLEN);
            }
        }
    }
    __syncthreads();
    if (!s.ok) return;  // the whole cluster

    Row w;
    w.p = g.target_probs + (long long)s.from * g.target_stride;
    w.q = s.rejected && g.draft_probs ? g.draft_probs + (long long)s.from * g.draft_stride : nullptr;
    w.point = s.rejected && !g.draft_probs ? s.point : -1;
    // This warp's stretch: the cluster's warps in order.
    const long long at = (long long)(rank * kWarps + warp) * stretch;
    const int i0 = at < g.vocab ? (int)at : g.vocab;
    const int i1 = at + stretch < g.vocab ? (int)at + stretch : g.vocab;

    for (int round = 0;; ++round) {
        const u64 mine = warp_sum(lane_sum<VEC>(w, i0, i1, lane));
        if (lane == 0) s.warp_total[warp] = mine;
        cluster_sync();
        // Every warp adds up the sums before its own, and all: a lane a warp of the cluster, twice.
        u64 before = 0, all = 0;
        for (uint32_t k = lane; k < cs * kWarps; k += 32) {
            const u64 x = peer_word(&s.warp_total[k % kWarps], k / kWarps);
            all += x;
            if (k < rank * kWarps + warp) before += x;
        }
        before = warp_sum(before);
        all = warp_sum(all);
        cluster_sync();  // nobody writes its sums again, or leaves, before all have read them
        if (all == 0) {
            if (round == 0 && (w.q || w.point >= 0)) {  // p <= q everywhere: the next token comes from p
                w.q = nullptr;
                w.point = -1;
                continue;
            }
            if (rank == 0 && tid == 0) {
                next_ids[r] = -1;
                if (g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_TOKEN);
            }
            return;
        }
        const float us = g.u_sample[r];
        const u64 u = us > 0.f ? min(__float2ull_rz(us * 0x1p31f), (u64)0x7fffffff) : 0;
        const u64 border = __umul64hi(u, all) << 33 | u * all >> 31;  // floor(u all / 2^31)
        if (border < before || border >= before + mine) return;
        // The token is in this warp's stretch: the first at which the running sum passes the border.
        u64 sum = before;
        for (int b = i0; b < i1; b += 32 * 8) {
            u64 x[8], part = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = b + lane * 8 + e;
                x[e] = i < i1 ? w.weight(i, w.p[i], w.q ? w.q[i] : 0.f) : 0;
                part += x[e];
            }
            u64 incl = part;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            const unsigned m = __ballot_sync(0xffffffffu, sum + incl > border);
            if (m) {
                if (lane == __ffs(m) - 1) {
                    u64 c = sum + incl - part;
                    int i = b + lane * 8;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        c += x[e];
                        if (c <= border) ++i;
                    }
                    next_ids[r] = i;
                }
                return;
            }
            sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        return;
    }
}

}  // namespace

cudaError_t launch_sample(const gdn_sample &g, long long n_tok, int32_t *accepted, int32_t *next_ids,
                          cudaStream_t stream) {
    // Blocks of a request: as many as keep a tile or two for every warp, and the GPU's SMs
    // to eight blocks each.
    int cs = 1;
    while (cs < kMaxCluster && 2ll * cs * g.batch <= 8 * 152 && g.vocab > cs * kWarps * kTile) cs *= 2;
    const int warps = cs * kWarps;
    const int stretch = ((g.vocab + warps - 1) / warps + 3) / 4 * 4;
    const bool vec = (reinterpret_cast<uintptr_t>(g.target_probs) & 15) == 0 && g.target_stride % 4 == 0 &&
                     (!g.draft_probs || ((reinterpret_cast<uintptr_t>(g.draft_probs) & 15) == 0 &&
                                         g.draft_stride % 4 == 0));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.batch * (long long)cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return vec ? cudaLaunchKernelEx(&cfg, sample_kernel<true>, g, n_tok, stretch, accepted, next_ids)
               : cudaLaunchKernelEx(&cfg, sample_kernel<false>, g, n_tok, stretch, accepted, next_ids);
}

}  // namespace gdn
