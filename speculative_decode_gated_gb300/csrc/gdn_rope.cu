// Rotary positions of a step's queries and keys, with the append of its keys
// and values to the pages of the cache.
//
// Pair i of a head turns by the angle p * inv_freq[i].  A 32-bit product of a
// long context's position and a frequency has lost the angle's fraction (half
// a unit in the last place of 2^17 radians is 0.008), so the angle is kept in
// turns as a 64-bit fraction: F = inv_freq / (2 pi) * 2^64 modulo 2^64, from the
// frequency's 24 bits and 128 bits of 1 / (2 pi) in integers (the reduction of
// Payne and Hanek), and p * F modulo 2^64 is the
// position's fraction of a turn, off by less than p * 2^-64.  Its top 32 bits, as a
// float in [-1, 1) half turns, go to sincospif.
//
// Bound by memory: N (Hq + 2 Hkv) hd elements read once and written once.  One
// block of 128 threads per row: the row's loads depend on nothing but its number and go
// out first; its request, its place and its cosines and sines (computed once, into
// shared memory, for all heads) are found while they fly.  A thread moves two
// 16-byte vectors of a head at a time, the two halves of eight (bf16) pairs, or two
// neighbours.
//
// Measured: 64 requests of 16 rows (32 + 2 * 8 heads of 128, bf16, 25 MB that the L2 holds)
// 4.9 to 5.4 us; a prompt of 5127 rows (16 + 2 * 4 heads of 256, bf16, 126 MB) 26 us, 4.8 TB/s,
// half the issue slots busy; a single row 3 us, all of it latency.
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 128;  // head_dim / 2 at most: one a thread
static_assert(kMaxPairs <= kThreads, "");
constexpr int kUnroll = 4;      // vectors pairs in flight per thread

template <typename T>
struct Vec;  // 16 bytes as floats
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void unpack(const uint4 &w, float *f) {
        f[0] = __uint_as_float(w.x);
        f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z);
        f[3] = __uint_as_float(w.w);
    }
    __device__ static uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void unpack(const uint4 &w, float *f) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[2 * e] = __uint_as_float(x[e] << 16);
            f[2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 pack(const float *f) {  // rounded once, to nearest even
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            x[e] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(x[0], x[1], x[2], x[3]);
    }
};

struct RopeArgs {
    AttnArgs a;
    const void *k_new, *v_new;
    long long k_stride, v_stride;
    void *k_pages, *v_pages;
    int rot, interleaved;
    float mscale;
    const float *inv_freq;
    const int32_t *positions;
    int slot_shift;  // log2 of the vector pairs of a head
};

// Turns per position, times 2^64, modulo 2^64.
__device__ __forceinline__ unsigned long long turns(float f) {
    const uint32_t b = __float_as_uint(f);
    const unsigned long long m = (b & 0x7FFFFFu) | 0x800000u;  // |f| = m 2^(64 - n)
    const int n = 64 + 150 - (int)((b >> 23) & 0xFFu);
    if (((b >> 23) & 0xFFu) == 0) return 0;  // zero (or too small to turn)
    // m * floor(2^128 / (2 pi)), of which the bits from n on
    constexpr unsigned long long hi = 0x28BE60DB9391054Aull, lo = 0x7F09D5F47D4D3770ull;
    const unsigned long long p0 = m * lo, c = __umul64hi(m, lo);
    const unsigned long long p1 = m * hi + c, p2 = __umul64hi(m, hi) + (p1 < c);
    unsigned long long F;
    if (n >= 128)
        F = n < 192 ? p2 >> (n - 128) : 0;
    else if (n > 64)
        F = p1 >> (n - 64) | p2 << (128 - n);
    else if (n == 64)
        F = p1;
    else
        F = n > 0 ? p0 >> n | p1 << (64 - n) : p0 << (n > -64 ? -n : 63);
    return b >> 31 ? 0 - F : F;
}

// cos and sin of p times as much.
__device__ __forceinline__ float2 turn(int p, unsigned long long per_position) {
    const unsigned long long phase = per_position * (unsigned long long)(long long)p;
    const float x = (float)(int)(phase >> 32) * 0x1p-31f;  // in half turns, [-1, 1]
    float2 cs;
    sincospif(x, &cs.y, &cs.x);
    return cs;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs g) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int VE = Vec<T>::N;
    __shared__ float2 cs[kMaxPairs];
    __shared__ int found;
    const AttnArgs &a = g.a;
    const int row = blockIdx.x, tid = threadIdx.x;

    const T *qs = static_cast<const T *>(a.q) + row * a.q_stride;
    const T *ks = static_cast<const T *>(g.k_new) + row * g.k_stride;
    const T *vs = static_cast<const T *>(g.v_new) + row * g.v_stride;

    const int slots = 1 << g.slot_shift;          // vector pairs of a head
    const int nr = g.rot / VE;                    // rotated vectors of a head (even)
    const int total = (a.Hq + 2 * a.Hkv) << g.slot_shift;
    uint4 w[kUnroll][2];

    // Vector pair i: its two sources and destinations, in elements from the head.
    auto place_of = [&](int i, int &head, int &v0, int &v1) {
        head = i >> g.slot_shift;
        const int s = i & (slots - 1);
        v0 = 2 * s;
        v1 = 2 * s + 1;
        if (!g.interleaved && head < a.Hq + a.Hkv && s < nr / 2) {
            v0 = s;
            v1 = s + nr / 2;
        }
    };
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = base + u * kThreads + tid;
            if (i >= total) break;
            int head, v0, v1;
            place_of(i, head, v0, v1);
            const T *src = head < a.Hq            ? qs + head * a.hd
                           : head < a.Hq + a.Hkv ? ks + (head - a.Hq) * a.hd
                                                 : vs + (head - a.Hq - a.Hkv) * a.hd;
            w[u][0] = __ldcs(reinterpret_cast<const uint4 *>(src + v0 * VE));
            w[u][1] = __ldcs(reinterpret_cast<const uint4 *>(src + v1 * VE));
        }
    };
    const float freq = tid < g.rot / 2 ? g.inv_freq[tid] : 0.f;  // a pair a thread
    load(0);
    const unsigned long long per_position = turns(freq);

    // The row's request.
    int r;
    if (a.cu_seqlens) {
        if (row == 0)  // one block reports bad requests, those without rows among them
            for (int i = tid; i < a.B; i += kThreads) load_request(a, i, true);
        if (tid == 0) found = -1;
        __syncthreads();
        for (int i = tid; i < a.B; i += kThreads)
            if (a.cu_seqlens[i] <= row && row < a.cu_seqlens[i + 1]) found = i;
        __syncthreads();
        r = found;
        if (r < 0) return;
    } else {
        r = row / a.max_T;
    }
    const AttnReq q = load_request(a, r, tid == 0);
    if (!q.ok) return;
    const int place = q.ctx + (row - q.row0);
    const int page = a.page_table[(long long)r * a.max_pages + (place >> a.page_shift)];
    const bool page_ok = page >= 0 && page < a.n_pages;

    T *qd = static_cast<T *>(a.o) + (long long)row * a.Hq * a.hd;
    const int in_page = place & ((1 << a.page_shift) - 1);
    const long long at = (long long)page * a.page_stride + (long long)in_page * a.hd;
    T *kd = static_cast<T *>(g.k_pages) + at;  // + head * page size * hd
    T *vd = static_cast<T *>(g.v_pages) + at;

    auto store = [&](int base) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = base + u * kThreads + tid;
            if (i >= total) break;
            int head, v0, v1;
            place_of(i, head, v0, v1);
            if (head < a.Hq + a.Hkv && v0 < nr) {
                float x[VE], y[VE];
                Vec<T>::unpack(w[u][0], x);
                Vec<T>::unpack(w[u][1], y);
                if (g.interleaved) {
#pragma unroll
                    for (int e = 0; e < VE; e += 2) {
                        const float2 c0 = cs[e / 2 * nr + v0], c1 = cs[e / 2 * nr + v1];
                        const float x0 = x[e], y0 = y[e];
                        x[e] = x0 * c0.x - x[e + 1] * c0.y;
                        x[e + 1] = x0 * c0.y + x[e + 1] * c0.x;
                        y[e] = y0 * c1.x - y[e + 1] * c1.y;
                        y[e + 1] = y0 * c1.y + y[e + 1] * c1.x;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float2 c = cs[e * (nr / 2) + v0];
                        const float x0 = x[e];
                        x[e] = x0 * c.x - y[e] * c.y;
                        y[e] = x0 * c.y + y[e] * c.x;
                    }
                }
                w[u][0] = Vec<T>::pack(x);
                w[u][1] = Vec<T>::pack(y);
            }
            T *dst;
            if (head < a.Hq) {
                dst = qd + head * a.hd;
            } else {
                if (!page_ok) continue;
                const bool is_k = head < a.Hq + a.Hkv;
                const long long h = is_k ? head - a.Hq : head - a.Hq - a.Hkv;
                dst = (is_k ? kd : vd) + ((h * a.hd) << a.page_shift);
            }
            *reinterpret_cast<uint4 *>(dst + v0 * VE) = w[u][0];
            *reinterpret_cast<uint4 *>(dst + v1 * VE) = w[u][1];
        }
    };

    const int pos = g.positions ? g.positions[row] : place;
    if (tid < g.rot / 2) {
        const float2 c = turn(pos, per_position);
        // pair e of a vector's pairs: the vectors side by side
        const int pairs = g.interleaved ? VE / 2 : VE, vectors = g.interleaved ? nr : nr / 2;
        cs[tid % pairs * vectors + tid / pairs] = make_float2(c.x * g.mscale, c.y * g.mscale);
    }
    if (!page_ok && tid == 0 && a.dev_err) atomicOr(a.dev_err, GDN_DEVERR_PAGE);
    __syncthreads();
    store(0);
    for (int base = kUnroll * kThreads; base < total; base += kUnroll * kThreads) {
        load(base);
        store(base);
    }
}

}  // namespace

cudaError_t launch_rope(const AttnArgs &a, const gdn_rope &rope, bool bf16, const void *k,
                        long long k_stride, const void *v, long long v_stride, void *k_pages,
                        void *v_pages, cudaStream_t stream) {
    RopeArgs g;
    g.a = a;
    g.k_new = k;
    g.v_new = v;
    g.k_stride = k_stride;
    g.v_stride = v_stride;
    g.k_pages = k_pages;
    g.v_pages = v_pages;
    g.rot = rope.rot_dim;
    g.interleaved = rope.interleaved;
    g.mscale = rope.mscale;
    g.inv_freq = rope.inv_freq;
    g.positions = rope.positions;
    g.slot_shift = 0;
    const int pairs = a.hd / (bf16 ? 8 : 4) / 2;
    while ((1 << g.slot_shift) < pairs) ++g.slot_shift;
    if (a.n_tok == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n_tok);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return bf16 ? cudaLaunchKernelEx(&cfg, rope_kernel<__nv_bfloat16>, g)
                : cudaLaunchKernelEx(&cfg, rope_kernel<float>, g);
}

}  // namespace gdn
