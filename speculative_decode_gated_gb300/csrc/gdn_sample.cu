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
// A cluster of CS blocks takes a request, each warp of it a stretch of the row in kSubs parts:
// first the sums of all parts, then, by these, the one warp whose part holds the token reads
// that part again (from L2) for the place.  64 requests of 128000 ids take 18 us (48% of the copy's
// rate: the drafts' own loads, the sums' exchange and the second look are latencies), one of 32000 5.4 us.
//
// A float x in [0, 1] in units, without a conversion to 64 bits (whose instruction took most
// of the time: 56 us for 64 requests and 128000 ids, 34 us with shifts of the significand):
// the last place of x + 2, rounded down, is 2^-22, and that of what is left plus 2^-21 is 2^-44,
// so the sums' bits hold the leading and the following 22 bits of x, and differences of p's and
// q's bits those of p - q (leading and following ones apart, each with its sign).
#include <cstdint>

#include "gdn_device.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kTile = 512;  // ids that a warp takes at a time, 16 a lane
constexpr int kSubs = 8;    // parts of a warp's stretch, whole tiles

using u64 = unsigned long long;

// The weights of one request's row: p, or max(p - q, 0).
struct Row {
    const float *p, *q;  // q = NULL: all of p
    int point;           // the id of a looked-up draft that did not stay (q is 1 there), or -1
};

// Two values' sums with 2 and, of what that leaves, with 2^-21, rounded down.
struct Bits {
    uint32_t hi[2], lo[2];
};
__device__ __forceinline__ Bits bits_of(float x, float y) {  // in [0, 1]
    float2 big, rest;
    Bits b;
    asm("{\n .reg .b64 v, t, m, one;\n mov.b64 v, {%2, %3};\n mov.b64 m, {%4, %4};\n"
        " add.rz.f32x2 t, v, m;\n mov.b64 {%0, %1}, t;\n}\n"
        : "=f"(big.x), "=f"(big.y)
        : "f"(x), "f"(y), "f"(2.f));
    asm("{\n .reg .b64 v, t, m, one;\n mov.b64 v, {%2, %3};\n mov.b64 t, {%4, %5};\n mov.b64 m, {%6, %6};\n"
        " mov.b64 one, {%7, %7};\n add.rn.f32x2 t, t, m;\n fma.rn.f32x2 t, t, one, v;\n"  // both exact
        " mov.b64 m, {%8, %8};\n add.rz.f32x2 t, t, m;\n mov.b64 {%0, %1}, t;\n}\n"
        : "=f"(rest.x), "=f"(rest.y)
        : "f"(x), "f"(y), "f"(big.x), "f"(big.y), "f"(-2.f), "f"(-1.f), "f"(0x1p-21f));
    b.hi[0] = __float_as_uint(big.x);
    b.hi[1] = __float_as_uint(big.y);
    b.lo[0] = __float_as_uint(rest.x);
    b.lo[1] = __float_as_uint(rest.y);
    return b;
}

// Sums of weights, the leading and the following 22 bits apart; of 16 weights each fits 32 bits.
struct Sum {
    uint32_t hi = 0, lo = 0;
    // Two ids' p and q as they are.  saturate takes NaN and below 0 to 0, above 1 to 1.
    __device__ __forceinline__ void add(float x0, float x1, float y0, float y1) {
        x0 = __saturatef(x0);
        x1 = __saturatef(x1);
        y0 = __saturatef(y0);
        y1 = __saturatef(y1);
        const Bits x = bits_of(x0, x1), y = bits_of(y0, y1);
        if (x0 > y0) {  // else q has at least p's units
            hi += x.hi[0] - y.hi[0];
            lo += x.lo[0] - y.lo[0];
        }
        if (x1 > y1) {
            hi += x.hi[1] - y.hi[1];
            lo += x.lo[1] - y.lo[1];
        }
    }
    __device__ __forceinline__ void add(float x0, float x1) {  // q = 0
        const Bits x = bits_of(__saturatef(x0), __saturatef(x1));
        hi += x.hi[0] + x.hi[1] - 0x80000000u;   // of 2 twice
        lo += x.lo[0] + x.lo[1] - 0x6A000000u;   // of 2^-21 twice
    }
    __device__ __forceinline__ u64 units() const {
        return ((u64)hi << 22) + (u64)(long long)(int)lo;
    }
};

// This lane's share of the weights of ids [at, end), a tile at a time: id (u, e) of its 16 is at +
// 128 u + 4 lane + e, or, without vectors, at + 32 (4 u + e) + lane.
template <bool VEC>
__device__ __forceinline__ int id_of(int at, int lane, int u, int e) {
    return VEC ? at + 128 * u + 4 * lane + e : at + 32 * (4 * u + e) + lane;
}
template <bool VEC, bool WHOLE>  // WHOLE: all ids are of the part; else those outside count as 0
__device__ __forceinline__ void load_tile(const float *row, int at, int first, int end, int lane, float (*x)[4]) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = id_of<VEC>(at, lane, u, 0);
        if (VEC && (WHOLE || (i >= first && i + 4 <= end))) {
            const float4 y = __ldg(reinterpret_cast<const float4 *>(row + i));
            x[u][0] = y.x;
            x[u][1] = y.y;
            x[u][2] = y.z;
            x[u][3] = y.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = id_of<VEC>(at, lane, u, e);
                x[u][e] = WHOLE || (k >= first && k < end) ? __ldg(row + k) : 0.f;
            }
        }
    }
}
template <bool VEC, bool WHOLE>
__device__ __forceinline__ u64 tile_sum(const Row &w, int at, int first, int end, int lane) {
    float x[4][4], y[4][4];
    Sum t;
    load_tile<VEC, WHOLE>(w.p, at, first, end, lane, x);
    if (w.q) {
        load_tile<VEC, WHOLE>(w.q, at, first, end, lane, y);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            t.add(x[u][0], x[u][1], y[u][0], y[u][1]);
            t.add(x[u][2], x[u][3], y[u][2], y[u][3]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            t.add(x[u][0], x[u][1]);
            t.add(x[u][2], x[u][3]);
        }
    }
    return t.units();
}
template <bool VEC>
__device__ __forceinline__ u64 lane_sum(const Row &w, int at, int end, int lane) {
    const int first = max(at, 0);
    u64 sum = 0;
    for (; at < end; at += kTile)
        sum += at >= 0 && at + kTile <= end ? tile_sum<VEC, true>(w, at, first, end, lane)
                                            : tile_sum<VEC, false>(w, at, first, end, lane);
    if (lane == 0 && w.point >= first && w.point < end) {
        Sum t;
        t.add(w.p[w.point], 0.f);
        sum -= t.units();  // what q has there; a share may be below 0, the sum over lanes is not
    }
    return sum;
}

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
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
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
    u64 warp_total[kWarps], sub[kWarps][kSubs];
    int accepted, from;  // rows kept; the row of p (and q) the next token comes from
    int point, rejected, ok;
};

__global__ void __launch_bounds__(kThreads, 4)
    sample_kernel(const gdn_sample g, long long n_tok, int tiles, int32_t *accepted, int32_t *next_ids) {
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
    // This warp's stretch of the row, `tiles` tiles: the cluster's warps in order.  Tiles begin where p
    // is 16-byte aligned, `off` elements before a multiple of 4, so a row of any length is read in
    // vectors; q's row is too where it lies as p's does.
    const int off = (int)(reinterpret_cast<uintptr_t>(w.p) >> 2) & 3;
    const bool vec = !w.q || ((int)(reinterpret_cast<uintptr_t>(w.q) >> 2) & 3) == off;
    const int of_part = (tiles + kSubs - 1) / kSubs;  // tiles
    auto begin = [&](int k) {
        const int i = ((int)(rank * kWarps + warp) * tiles + min(k * of_part, tiles)) * kTile - off;
        return i < g.vocab ? i : g.vocab;
    };
    const float us = g.u_sample[r];
    auto locate = [&](u64 border, u64 before) {
        // The token is in this warp's stretch, in the part at which the running sum passes the border;
        // there, 8 ids a lane at a time, at the first id that does.
        __syncwarp();
        u64 sum = before;
        int k = 0;
        for (; (k + 1) * of_part < tiles && sum + s.sub[warp][k] <= border; ++k) sum += s.sub[warp][k];
        const int end = begin(k + 1);
        for (int at = begin(k); at < end; at += 256) {
            u64 x[8], all_of = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int i = at + lane * 8 + e;
                Sum one;
                if (i >= 0 && i < end)
                    one.add(w.p[i], 0.f, w.q ? w.q[i] : i == w.point ? 1.f : 0.f, 0.f);
                x[e] = one.units();
                all_of += x[e];
            }
            u64 incl = all_of;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += y;
            }
            const unsigned m = __ballot_sync(0xffffffffu, sum + incl > border);
            if (m) {
                if (lane == __ffs(m) - 1) {
                    u64 c = sum + incl - all_of;
                    int i = at + lane * 8;
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
    };
    for (int round = 0;; ++round) {
        u64 mine = 0;
#pragma unroll 1
        for (int k = 0; k * of_part < tiles; ++k) {
            const u64 x = warp_sum(vec ? lane_sum<true>(w, begin(k), begin(k + 1), lane)
                                       : lane_sum<false>(w, begin(k), begin(k + 1), lane));
            if (lane == 0) s.sub[warp][k] = x;
            mine += x;
        }
        if (lane == 0) s.warp_total[warp] = mine;
        cluster_arrive();
        cluster_wait();
        // Every warp adds up the sums before its own, and all: a lane a warp of the cluster, twice.
        u64 before = 0, all = 0;
        for (uint32_t k = lane; k < cs * kWarps; k += 32) {
            const u64 x = peer_word(&s.warp_total[k % kWarps], k / kWarps);
            all += x;
            if (k < rank * kWarps + warp) before += x;
        }
        before = warp_sum(before);
        all = warp_sum(all);
        cluster_arrive();  // nobody writes its sums again, or leaves, before all have read them
        if (all == 0) {
            cluster_wait();
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
        const u64 u = us > 0.f ? min(__float2ull_rz(us * 0x1p31f), (u64)0x7fffffff) : 0;
        const u64 border = __umul64hi(u, all) << 33 | u * all >> 31;  // floor(u all / 2^31)
        if (border >= before && border < before + mine) locate(border, before);
        cluster_wait();
        return;
    }
}

}  // namespace

cudaError_t launch_sample(const gdn_sample &g, long long n_tok, int32_t *accepted, int32_t *next_ids,
                          cudaStream_t stream) {
    // Blocks of a request: as many as keep a tile for every warp and are resident at once, four an
    // SM (200 requests of 100003 ids, 23 to 25 us with two blocks each, 28 with four).
    int cs = 1;
    while (cs < kMaxCluster && 2ll * cs * g.batch <= 4 * 152 && g.vocab > cs * kWarps * kTile) cs *= 2;
    // (3 ids more than there are: where a row begins within 16 bytes)
    const int tiles = ((g.vocab + 3 + kTile - 1) / kTile + cs * kWarps - 1) / (cs * kWarps);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel, g, n_tok, tiles, accepted, next_ids);
}

}  // namespace gdn
