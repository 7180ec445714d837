// The next step's lengths, pages, row offsets, slots and positions (gdn_plan_pages; the
// rules are in gdn.h).
//
// Whole numbers and little work: bound by latency.  One cluster of blocks does it in one launch.
// A thread takes a request, a block 1024 of them at a time, and every block of the cluster
// adds up all requests for itself (their few words come from L2; handing sums around would
// take longer).  What there is to move (pages that go back, pages that come, rows) is numbered
// through and spread over all threads of the cluster, each finding the request of its number by
// bisection in the block's running sums, so one long prompt takes no longer than many short ones.
//   pass 1  what goes back, summed over all requests, and its pages written behind the list;
//   pass 2  with the list's length known: who gets pages, and these into the page table;
//   pass 3  lengths, held pages and row offsets: the first block alone, after all have read
//           the arrays that these may overwrite.
// Slots and positions follow in the same launch while few rows are possible, else in a
// launch of their own over the whole GPU.  64 requests of 16 rows take 6 us, 1000 requests of up to
// 2000 rows (a million slots) 23 us, half of it the second launch.
#include <cstdint>

#include "gdn_device.cuh"
#include "gdn_launch.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCluster = 8;
// Rows of slots and positions that the planning launch writes itself.  8192 rows of 64 requests take 10 us so
// and 16 in two launches; 16384 rows 12 and 14.
constexpr int kInline = 8192;

// What one request wants.
struct Want {
    int len;    // its length in the next step
    int rows;   // rows, if it gets its pages
    int held;   // pages held now
    int need;   // pages wanted
    int err;    // error bits
    bool stay;  // nothing moves: bad arguments
};

__device__ __forceinline__ Want want_of(const gdn_pages &g, int shift, int r) {
    Want w;
    const int kv = g.kv_len[r], acc = g.accepted ? g.accepted[r] : 0, rows = g.rows ? g.rows[r] : g.max_T;
    const bool done = g.done && g.done[r] != 0;
    w.held = g.held[r];
    w.err = 0;
    if (w.held < 0 || w.held > g.max_pages || (!done && kv < 0)) w.err |= GDN_DEVERR_KV_LEN;
    if (!done && !w.err && (acc < 0 || (long long)kv + acc > ((long long)w.held << shift)))
        w.err |= GDN_DEVERR_ACCEPTED;
    if (!done && (rows < 0 || rows > g.max_T)) w.err |= GDN_DEVERR_SEQLEN;
    w.stay = w.err != 0;
    w.len = w.stay ? kv : done ? 0 : kv + acc;
    w.rows = w.stay || done ? 0 : rows;
    if (!w.stay && (long long)w.len + w.rows > ((long long)g.max_pages << shift)) {
        w.err |= GDN_DEVERR_KV_LEN;
        w.rows = 0;
    }
    w.need = w.stay ? w.held : (int)(((long long)w.len + w.rows + g.page_size - 1) >> shift);
    return w;
}

// Nothing to do for threads behind the last request.
__device__ __forceinline__ Want nobody() { return Want{0, 0, 0, 0, 0, true}; }

struct Shared {
    uint32_t warp_sum[2][kWarps];
    uint32_t before[kThreads + 1];  // running sums of what the tile's requests move
    int from[kThreads];             // first column (first position) of each
    uint32_t base[kThreads];        // its place in the free list (its rows' number)
};

// Exclusive sum over the block's threads, and the sum of all.  A call in between of the other
// parity keeps two calls' words apart.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *warp_sum, uint32_t &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t w = warp_sum[lane], wi = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, wi, d);
        if (lane >= d) wi += y;
    }
    all = __shfl_sync(0xffffffffu, wi, 31);
    const uint32_t out = __shfl_sync(0xffffffffu, wi - w, warp) + incl - x;
    __syncthreads();
    return out;
}

// The entry e of [0, n) with before[e] <= m < before[e + 1]; m < before[n].
__device__ __forceinline__ int entry_of(const uint32_t *before, int n, uint32_t m) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= m)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                     : "memory");
}

// Row `n` of the step: a row of request r, at place `place`.
__device__ __forceinline__ void write_row(const gdn_pages &g, int shift, long long n, int r, int place) {
    if (g.slots) {
        const long long page = __ldcg(g.page_table + (long long)r * g.max_pages + (place >> shift));
        g.slots[n] = (page << shift) + (place & (g.page_size - 1));
    }
    if (g.positions) g.positions[n] = place;
}

__global__ void __launch_bounds__(kThreads) pages_kernel(const gdn_pages g, int shift, int rows_here) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Shared s;
    const int tid = threadIdx.x, B = g.batch;
    const int rank = blockIdx.x, all_threads = gridDim.x * kThreads, me = rank * kThreads + tid;
    const bool many = B > kThreads;  // more than one tile: a thread's request is read again in each pass
    Want w = tid < B ? want_of(g, shift, tid) : nobody();
    const int count = *g.free_count;

    // Pass 1.
    uint32_t back_all = 0;
    const bool count_ok = count >= 0 && count <= g.n_pages;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        if (b0 > 0) w = b0 + tid < B ? want_of(g, shift, b0 + tid) : nobody();
        const uint32_t back = w.need < w.held ? w.held - w.need : 0;
        uint32_t all;
        s.before[tid] = block_scan(back, s.warp_sum[0], all);
        s.from[tid] = w.need;
        if (tid == 0) s.before[kThreads] = all;
        __syncthreads();
        if (count_ok)
            for (uint32_t m = me; m < all; m += all_threads) {
                const int e = entry_of(s.before, kThreads, m);
                const long long to = (long long)count + back_all + m;
                if (to < g.n_pages)
                    g.free_pages[to] = __ldcg(g.page_table + (long long)(b0 + e) * g.max_pages +
                                              s.from[e] + (int)(m - s.before[e]));
            }
        back_all += all;
        __syncthreads();
    }
    const bool list_ok = count_ok && (long long)count + back_all <= g.n_pages;
    const uint32_t available = list_ok ? count + back_all : 0;
    if (!list_ok && rank == 0 && tid == 0 && g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_PAGE);
    cluster_sync();  // what went back is in the list

    // Pass 2 (and, with one tile, pass 3 from the same registers).
    uint32_t more_all = 0, taken = 0, rows_all = 0;
    auto grant = [&](uint32_t more, uint32_t before) {
        return list_ok && (more == 0 || before + more <= available);
    };
    bool granted = false;
    uint32_t row0 = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        if (many) w = b0 + tid < B ? want_of(g, shift, b0 + tid) : nobody();
        const uint32_t more = w.need > w.held ? w.need - w.held : 0;
        uint32_t all, moved;
        const uint32_t before = more_all + block_scan(more, s.warp_sum[0], all);
        // in 32 bits: held and wanted pages are entries of the page table, at most 2^31 - 1
        granted = grant(more, before);
        const uint32_t comes = granted ? more : 0;
        s.before[tid] = block_scan(comes, s.warp_sum[1], moved);
        s.from[tid] = w.held;
        s.base[tid] = before;
        if (tid == 0) s.before[kThreads] = moved;
        __syncthreads();
        for (uint32_t m = me; m < moved; m += all_threads) {
            const int e = entry_of(s.before, kThreads, m);
            const uint32_t i = m - s.before[e];
            g.page_table[(long long)(b0 + e) * g.max_pages + s.from[e] + (int)i] =
                __ldcg(g.free_pages + (available - 1 - (s.base[e] + i)));
        }
        more_all += all;
        taken += moved;
        __syncthreads();
    }
    cluster_sync();  // all have read what pass 3 may overwrite, and the page table is written

    // Pass 3.
    more_all = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int r = b0 + tid;
        if (many) {
            if (rank != 0) break;  // the others would read what the first block writes
            w = r < B ? want_of(g, shift, r) : nobody();
            const uint32_t more = w.need > w.held ? w.need - w.held : 0;
            uint32_t all;
            const uint32_t before = more_all + block_scan(more, s.warp_sum[0], all);
            more_all += all;
            granted = grant(more, before);
        }
        uint32_t all;
        const int rows = granted ? w.rows : 0;
        row0 = rows_all + block_scan(rows, s.warp_sum[1], all);
        rows_all += all;
        if (rank == 0 && r < B) {
            int err = w.err;
            if (list_ok && !granted) err |= GDN_DEVERR_NO_PAGES;
            // (a bad list: nothing moves)
            g.kv_len_out[r] = list_ok ? w.len : g.kv_len[r];
            g.held_out[r] = granted ? w.need : w.held;
            g.cu_seqlens[r] = (int)row0;
            if (r == B - 1) g.cu_seqlens[B] = (int)rows_all;
            if ((g.slots || g.positions) && rows_all > g.max_rows && r == B - 1) err |= GDN_DEVERR_SEQLEN;
            if (err && g.dev_err) atomicOr(g.dev_err, err);
        }
        if (rows_here) {  // one tile
            s.before[tid] = row0;
            s.from[tid] = w.len;
            if (tid == 0) s.before[kThreads] = rows_all;
        }
    }
    if (rank == 0 && tid == 0) *g.free_count_out = list_ok ? (int)(available - taken) : count;
    if (!rows_here) return;
    __syncthreads();
    for (uint32_t n = me; n < rows_all && n < g.max_rows; n += all_threads) {
        const int r = entry_of(s.before, kThreads, n);
        write_row(g, shift, n, r, s.from[r] + (int)(n - s.before[r]));
    }
}

// Slots and positions of many rows: a warp takes kRun rows in a row, finds the requests of
// the first and the last, and bisects between these.
constexpr int kRun = 256;
__global__ void __launch_bounds__(256) slots_kernel(const gdn_pages g, int shift) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long all = g.cu_seqlens[g.batch];
    const long long rows = all < g.max_rows ? all : g.max_rows;
    const long long step = (long long)gridDim.x * 8 * kRun;
    for (long long n0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kRun; n0 < rows; n0 += step) {
        auto find = [&](int lo, int hi, long long n) {  // lo <= its request < hi
            while (hi - lo > 1) {
                const int mid = lo + ((hi - lo) >> 1);
                if (g.cu_seqlens[mid] <= n)
                    lo = mid;
                else
                    hi = mid;
            }
            return lo;
        };
        const long long n1 = n0 + kRun < rows ? n0 + kRun : rows;
        const int end = find(0, g.batch, lane == 0 ? n0 : n1 - 1);
        const int first = __shfl_sync(0xffffffffu, end, 0), last = __shfl_sync(0xffffffffu, end, 1);
#pragma unroll 2
        for (long long n = n0 + lane; n < n1; n += 32) {
            const int r = first == last ? first : find(first, last + 1, n);
            write_row(g, shift, n, r, g.kv_len_out[r] + (int)(n - g.cu_seqlens[r]));
        }
    }
}

}  // namespace

cudaError_t launch_pages(const gdn_pages &g, cudaStream_t stream) {
    const long long rows = (long long)g.batch * g.max_T;
    const bool wanted = g.slots || g.positions;
    int shift = 0;
    while (1 << shift < g.page_size) ++shift;
    const bool here = wanted && rows <= kInline && g.batch <= kThreads;
    cudaLaunchConfig_t cfg = {};
    // One block suffices where a thread has a few numbers at most to move: up to 1024 rows it takes what
    // eight take, 4096 rows of 64 requests 14 us for 10, 8192 rows 18 for 10.
    const int cs = rows <= 4096 && g.batch <= 512 ? 1 : kCluster;
    cfg.gridDim = dim3(cs);
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, pages_kernel, g, shift, here ? 1 : 0);
    if (e != cudaSuccess || !wanted || here || rows == 0) return e;
    const long long runs = ((rows < g.max_rows ? rows : g.max_rows) + kRun - 1) / kRun;
    if (runs == 0) return e;
    cfg.gridDim = dim3((unsigned)((runs + 7) / 8 < 8 * 152 ? (runs + 7) / 8 : 8 * 152));
    cfg.blockDim = dim3(256);
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, slots_kernel, g, shift);
}

}  // namespace gdn
