// Linear attention of drafts on the tensor cores (mma.sync): outputs only, bf16, dk 64 or 128, dv a
// multiple of 64, fewer rows than the prompts' kernel takes.
//
// The state before the drafts stays as it is, so all of a request's rows read the same one:
//     o_i = scale (d(i, -1) S^T q_i + sum_{j <= i} d(i, j) (q_i . k_j) v_j)
// Bound by the states' bytes (64 KB a head of 128 x 128).  A block goes through units (request,
// head, 64 value columns): one warp asks the TMA engine for their states and rows (128-byte swizzle, two
// units' worth of shared memory), one works out their decays, and eight each take 8 columns of a unit
// from there to o, so none waits for another.  A product has 16 rows of a
// draft, so few rows cost as much as 16.  The state enters as two bf16 terms, off by 2^-17 of itself,
// and so do the weights d(i, j) (q_i . k_j), which are operands of the values' product just where their
// own product left them; q, k and v are bf16 already, and sums are float32.  16 rows of 64 requests and
// 32 heads of 128 take 34 us, 69% of the copy's rate (78 on CUDA cores): the warps' own work on a unit, 40%
// of the issue slots, is what the next unit's copies do not hide.
#include <cstdint>

#include "gdn_launch.h"
#include "gdn_linear.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;  // that compute, 8 columns each; one that loads, and one for the decays
constexpr int CV = 8 * kWarps;

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

// A unit: its rows (T < 0: no more units), head, first value column, and its state's first row in the pool.
struct Work {
    int T, row0, h, c0, row;
};

// NG groups of 16 rows.
template <int DK, int NG>
struct Tiles {
    static constexpr int T = 16 * NG;
    static constexpr int BUFFERS = 2;
    struct Unit {
        float state[2][DK][32];
        __nv_bfloat16 q[DK / 64][T][64], k[DK / 64][T][64], v[T][64];
    } unit[BUFFERS];
    struct Decays {
        alignas(8) float d[T][T + 2];  // d(i, j)
        float from[T];                 // d(i, -1)
    } decays[BUFFERS];
    float g[T];
    Work work[BUFFERS];
    int dead;  // a wait gave up
    unsigned long long full[BUFFERS], decayed[BUFFERS], free[BUFFERS];  // copies there; decays there; both done with
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

__device__ __forceinline__ void ldmatrix4(uint32_t *x, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix2_trans(uint32_t *x, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];\n"
                 : "=r"(x[0]), "=r"(x[1])
                 : "r"(at)
                 : "memory");
}
// 16 bytes c of row r of a tile whose rows have 128.
__device__ __forceinline__ uint32_t chunk(uint32_t tile, int r, int c) { return tile + r * 128 + ((c ^ (r & 7)) << 4); }

// Two bf16 values: whether one is not finite; the same with 0 for such.
__device__ __forceinline__ bool not_finite(uint32_t x) {
    return (x & 0x7F80u) == 0x7F80u || (x & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t finite_part(uint32_t x) {
    return ((x & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) | ((x & 0x7F800000u) == 0x7F800000u ? 0u : x & 0xFFFF0000u);
}
// Adds the values that are not finite in rows j0 to j0 + 15 of a tile (those below T), columns 8 warp on, to the
// warp's 16 rows of outputs from each one's own row on, by the weights' two terms.  (Rare, but not out of
// line: the weights would then go through memory in every product, 38 us where it is 34.2 so.)
__device__ __forceinline__ void add_not_finite(float *out, const uint32_t *W, const uint32_t *R, uint32_t vt, int j0,
                                               int T, int warp, int lane) {
    const int gr = lane >> 2, c = lane & 3;
#pragma unroll 1
    for (int j = 0; j < 16 && j0 + j < T; ++j) {
        const int from = 4 * gr + (j >> 1 & 3), n = j >> 3;  // the lane that has this row's weights
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // of output rows gr and gr + 8
            const uint32_t hi = __shfl_sync(0xffffffffu, n ? W[2 + i] : W[i], from);
            const uint32_t lo = __shfl_sync(0xffffffffu, n ? R[2 + i] : R[i], from);
            w[i] = j & 1 ? high(hi) + high(lo) : low(hi) + low(lo);
        }
        uint32_t v;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(chunk(vt, j0 + j, warp) + 4 * c) : "memory");
        const float x = low(v), y = high(v);
        const bool bad_x = (v & 0x7F80u) == 0x7F80u, bad_y = (v & 0x7F800000u) == 0x7F800000u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (gr + 8 * i < j) continue;
            if (bad_x) out[2 * i] = fmaf(w[i], x, out[2 * i]);
            if (bad_y) out[2 * i + 1] = fmaf(w[i], y, out[2 * i + 1]);
        }
    }
}

// The units of a block in order, `step` at a time; a unit's words are loaded a round before they are
// looked at.  One lane's answer is the warp's.
template <int DK>
struct Units {
    struct Place {
        unsigned r, h, s;
    };
    struct Words {
        int c0, c1, slot;
        Place p;
    };
    const LinearArgs &a;
    const unsigned units, slices, step;
    unsigned at;
    Place by, ahead;
    Words coming;

    __device__ __forceinline__ Units(const Launch &L)
        : a(L.a), units(L.units), slices(L.a.g.dv / CV), step(gridDim.x), at(blockIdx.x) {  // (at + step: below 2^31)
        by = place_of(step);
        ahead = place_of(at);
        coming = words_of(ahead);
    }
    __device__ __forceinline__ Place place_of(unsigned i) const {
        const unsigned unit = i / slices, H = a.g.heads;
        return Place{unit / H, unit % H, i - unit * slices};
    }
    __device__ __forceinline__ Words words_of(const Place &p) const {
        const gdn_linear &g = a.g;
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
    }
    // The next unit that has rows; T = -1 after the last.
    __device__ __forceinline__ Work next(bool report) {
        const gdn_linear &g = a.g;
        while (at < units) {
            const Words x = coming;
            at += step;
            ahead.s += by.s;
            ahead.h += by.h;
            ahead.r += by.r;
            if (ahead.s >= slices) {
                ahead.s -= slices;
                ++ahead.h;
            }
            if (ahead.h >= (unsigned)g.heads) {
                ahead.h -= g.heads;
                ++ahead.r;
            }
            coming = words_of(ahead);
            LinearUnit u;
            if (linear_words(a, x.c0, x.c1, x.slot, (int)x.p.h, u, report))
                return Work{u.T, u.row0, (int)x.p.h, (int)x.p.s * CV,
                            (x.slot * g.heads + (int)x.p.h) * DK};  // (rows of the pool: below 2^31)
        }
        return Work{-1, 0, 0, 0, 0};
    }
};

// The warp that loads the units' states and rows.
template <int DK, int NG>
__device__ __forceinline__ void load_role(const Launch &L, Tiles<DK, NG> &s, int lane) {
    constexpr uint32_t kBytes = DK * CV * 4 + Tiles<DK, NG>::T * (2 * DK + CV) * 2;
    const gdn_linear &g = L.a.g;
    Units<DK> units(L);
    Ring<Tiles<DK, NG>::BUFFERS> ring;
    uint32_t issued = 0;
    for (;; ring.next()) {
        const Work w = units.next(lane == 0);
        if (!wait(bar(s.free[ring.slot]), ring.parity ^ 1, &s.dead)) break;
        ++issued;
        const uint32_t full = bar(s.full[ring.slot]);
        auto &to = s.unit[ring.slot];
        if (lane == 0) {
            s.work[ring.slot] = w;
            if (w.T < 0) {
                arrive(full);
            } else {
                arrive_expect(full, kBytes);
                for (int x = 0; x < 2; ++x) tma(to.state[x], &L.pool, w.c0 + 32 * x, w.row, full);
                const int col = w.h / L.a.group * DK;
                for (int x = 0; x < DK / 64; ++x) {
                    tma(to.q[x], &L.q, col + 64 * x, w.row0, full);
                    tma(to.k[x], &L.k, col + 64 * x, w.row0, full);
                }
                tma(to.v, &L.v, w.h * g.dv + w.c0, w.row0, full);
            }
        }
        __syncwarp();
        if (w.T < 0) break;
    }
    if (lane == 0)
        wait_copies<Tiles<DK, NG>::BUFFERS>(
            issued, [&](uint32_t slot, uint32_t parity) { wait_parity(bar(s.full[slot]), parity); });
}

// The warp that works out their decays.
template <int DK, int NG>
__device__ __forceinline__ void decay_role(const Launch &L, Tiles<DK, NG> &s, int lane) {
    constexpr int T = Tiles<DK, NG>::T, N = (T + 31) / 32;
    const gdn_linear &g = L.a.g;
    Units<DK> units(L);
    Ring<Tiles<DK, NG>::BUFFERS> ring;
    float log[N];
    auto load = [&](const Work &w) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            log[i] = 32 * i + lane < w.T
                         ? ld_early(g.log_decay + (long long)(w.row0 + 32 * i + lane) * g.decay_stride + w.h)
                         : 0.f;
    };
    Work w = units.next(false);
    load(w);
    for (;; ring.next()) {
        const int rows = w.T;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (32 * i + lane < T) s.g[32 * i + lane] = log[i];
        __syncwarp();
        if (rows >= 0) {
            w = units.next(false);
            load(w);
        }
        if (!wait(bar(s.free[ring.slot]), ring.parity ^ 1, &s.dead)) return;
        auto &to = s.decays[ring.slot];
        // Row i's: sums from its end on.  Up to 16 rows: a lane a row (l), two sums at a time.
        if (NG == 1 && rows > 0) {
            const int l = lane & 15;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = 2 * k + (lane >> 4);
                float sum = l <= i ? s.g[l] : 0.f;
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) {
                    const float z = __shfl_down_sync(0xffffffffu, sum, d, 16);
                    if (l + d <= i) sum += z;
                }
                const float d = expf(sum);  // of rows l to i: d(i, l - 1)
                if (l == 0) {
                    to.from[i] = d;
                    to.d[i][i] = 1.f;
                } else if (l <= i) {
                    to.d[i][l - 1] = d;
                }
            }
        } else {
            for (int l = lane; l < rows; l += 32) {  // down column l - 1
                float sum = 0.f;
                to.d[l][l] = 1.f;
                for (int i = l; i < rows; ++i) {
                    sum += s.g[i];
                    const float d = expf(sum);
                    if (l == 0)
                        to.from[i] = d;
                    else
                        to.d[i][l - 1] = d;
                }
            }
        }
        arrive_warp(bar(s.decayed[ring.slot]));
        if (rows < 0) return;
    }
}

template <int DK, int NG>
__global__ void __launch_bounds__(32 * (kWarps + 2), 2) drafts_kernel(const __grid_constant__ Launch L) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ __align__(1024) unsigned char raw[];
    constexpr int NB = Tiles<DK, NG>::BUFFERS;
    Tiles<DK, NG> &s = *reinterpret_cast<Tiles<DK, NG> *>(raw);
    const gdn_linear &g = L.a.g;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gr = lane >> 2, c = lane & 3;
    if (tid == 0) {
        for (int i = 0; i < NB; ++i) {
            mbar_init(bar(s.full[i]), 1);
            mbar_init(bar(s.decayed[i]), 1);
            mbar_init(bar(s.free[i]), kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s.dead = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    if (warp >= kWarps) {
        if (warp == kWarps)
            load_role<DK, NG>(L, s, lane);
        else
            decay_role<DK, NG>(L, s, lane);
        return;
    }

    const int l7 = lane & 7, l8 = (lane >> 3) & 1, l16 = lane >> 4;
    Ring<NB> ring;
    for (;;) {
        if (!wait(bar(s.full[ring.slot]), ring.parity, &s.dead) ||
            !wait(bar(s.decayed[ring.slot]), ring.parity, &s.dead)) {  // they never came
            if (lane == 0 && g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_TIMEOUT);
            return;
        }
        const Work w = s.work[ring.slot];
        const int T = w.T;
        if (T < 0) return;
        const auto &in = s.unit[ring.slot];
        const auto &dec = s.decays[ring.slot];
        const uint32_t qt = smem_addr(in.q), kt = smem_addr(in.k), vt = smem_addr(in.v);
        // This lane's column of this warp's 8, in rows 16 st + 2c and so on of the state.
        const float *col = &in.state[warp >> 2][0][0] + (gr & 3);
        const int cc = 2 * (warp & 3) + (gr >> 2);
        auto element = [&](int row) { return col[row * 32 + 4 * (cc ^ (row & 7))]; };
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(L.a.o) + ((long long)w.row0 * g.heads + w.h) * g.dv + w.c0 +
                           8 * warp + 2 * c;

#pragma unroll 1
        for (int m = 0; 16 * m < T; ++m) {
            uint32_t A[DK / 16][4];
            float acc[2][4] = {};
#pragma unroll
            for (int st = 0; st < DK / 16; ++st) {
                ldmatrix4(A[st], chunk(qt + (st >> 2) * Tiles<DK, NG>::T * 128, 16 * m + l7 + 8 * l8,
                                       2 * (st & 3) + l16));
                const int row = 16 * st + 2 * c;
                const float x0 = element(row), x1 = element(row + 1), y0 = element(row + 8), y1 = element(row + 9);
                const uint32_t b0 = pack(x0, x1), b1 = pack(y0, y1);
                mma(acc[0], A[st], pack(x0 - low(b0), x1 - high(b0)), pack(y0 - low(b1), y1 - high(b1)));
                mma(acc[1], A[st], b0, b1);
            }
            // Rows gr and gr + 8 of the group.  (Of rows that are not there everything may be anything: it
            // stays in its row.)
            const int i0 = 16 * m + gr, i1 = i0 + 8;
            const float from0 = dec.from[i0], from1 = dec.from[i1];
            float out[4] = {(acc[0][0] + acc[1][0]) * from0, (acc[0][1] + acc[1][1]) * from0,
                            (acc[0][2] + acc[1][2]) * from1, (acc[0][3] + acc[1][3]) * from1};
            for (int l = 0; l <= m; ++l) {
                float own[2][4] = {};
#pragma unroll
                for (int st = 0; st < DK / 16; ++st) {
                    uint32_t b[4];
                    ldmatrix4(b, chunk(kt + (st >> 2) * Tiles<DK, NG>::T * 128, 16 * l + l7 + 8 * l16,
                                       2 * (st & 3) + l8));
                    mma(own[0], A[st], b[0], b[1]);
                    mma(own[1], A[st], b[2], b[3]);
                }
                uint32_t W[4], R[4];  // the weights' two terms
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int j = 16 * l + 8 * n + 2 * c;
                    const float2 d0 = *reinterpret_cast<const float2 *>(&dec.d[i0][j]);
                    const float2 d1 = *reinterpret_cast<const float2 *>(&dec.d[i1][j]);
                    const float w0 = j <= i0 ? own[n][0] * d0.x : 0.f, w1 = j < i0 ? own[n][1] * d0.y : 0.f;
                    const float w2 = j <= i1 ? own[n][2] * d1.x : 0.f, w3 = j < i1 ? own[n][3] * d1.y : 0.f;
                    W[2 * n] = pack(w0, w1);
                    W[2 * n + 1] = pack(w2, w3);
                    R[2 * n] = pack(w0 - low(W[2 * n]), w1 - high(W[2 * n]));
                    R[2 * n + 1] = pack(w2 - low(W[2 * n + 1]), w3 - high(W[2 * n + 1]));
                }
                uint32_t v[2];
                ldmatrix2_trans(v, chunk(vt, 16 * l + (lane & 15), warp));
                if (16 * l + 16 > T) {  // values that are not there: their weights are 0, they may be anything
                    const int j = 16 * l + 2 * c;
                    v[0] &= (j < T ? 0xFFFFu : 0u) | (j + 1 < T ? 0xFFFF0000u : 0u);
                    v[1] &= (j + 8 < T ? 0xFFFFu : 0u) | (j + 9 < T ? 0xFFFF0000u : 0u);
                }
                // A value that is not finite would reach rows before its own by their weight of 0, so it
                // leaves the product, and rows from its own on add it for themselves.
                const bool odd = l == m && __any_sync(0xffffffffu, not_finite(v[0]) || not_finite(v[1]));
                if (odd) {
                    v[0] = finite_part(v[0]);
                    v[1] = finite_part(v[1]);
                }
                mma(out, R, v[0], v[1]);
                mma(out, W, v[0], v[1]);
                if (odd) add_not_finite(out, W, R, vt, 16 * l, T, warp, lane);
            }
            const long long step = (long long)g.heads * g.dv;
            if (i0 < T) *reinterpret_cast<uint32_t *>(o + i0 * step) = pack(out[0] * g.scale, out[1] * g.scale);
            if (i1 < T) *reinterpret_cast<uint32_t *>(o + i1 * step) = pack(out[2] * g.scale, out[3] * g.scale);
        }
        arrive_warp(bar(s.free[ring.slot]));
        ring.next();
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
    constexpr int fit = 233472 / (smem + 1024), per_sm = fit < 2 ? fit : 2;
    static_assert(per_sm >= 1, "");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(L.units < 152 * per_sm ? L.units : 152 * per_sm);
    cfg.blockDim = dim3(32 * (kWarps + 2));
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
    return g.dtype == GDN_BF16 && (g.dk == 64 || g.dk == 128) && g.dv % CV == 0 && g.max_T > 1 &&
           g.max_T < kLinearTcRows &&
           g.pool_slots * g.heads * g.dk <= 0x7fffffffLL;  // the pool's rows are numbered in 32 bits
}

cudaError_t launch_linear_drafts(const LinearArgs &a, cudaStream_t stream) {
    if (a.g.dk == 64) return a.g.max_T <= 16 ? launch_one<64, 1>(a, stream) : launch_one<64, 3>(a, stream);
    return a.g.max_T <= 16 ? launch_one<128, 1>(a, stream) : launch_one<128, 3>(a, stream);
}

}  // namespace gdn
