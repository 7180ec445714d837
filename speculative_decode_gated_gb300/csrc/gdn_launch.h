// Host-side launchers of the kernels (internal to libgdn.so).
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "gdn_attn.cuh"
#include "gdn_device.cuh"
#include "gdn_linear.cuh"

namespace gdn {

// Recurrent kernel: dk in {32, 64, 128, 256}; dv a multiple of 32, <= 128 or a
// multiple of 128 up to 256; q/k/v bf16 or fp32; any max_T.
cudaError_t launch_recurrent(const Args &p, int mode, bool bf16, cudaStream_t stream);

// Chunked tensor-core kernel and its applicability.  One call covers n
// problems (layers) that share every request-level field; up to
// kChunkMaxLayers of them run in one launch, more are split into several.
constexpr int kChunkMaxLayers = 32;
bool chunk_supported(bool bf16, int dk, int dv, int max_T);
bool chunk_preferred(int max_T);
cudaError_t launch_chunk(const Args *layers, int n, int mode, cudaStream_t stream);

// Greedy accepted lengths (arguments already validated on the host).
cudaError_t launch_accept(int B, int max_T, const int32_t *cu_seqlens, long long n_tok,
                          const int32_t *draft, const int32_t *target, int32_t *accepted,
                          int32_t *dev_err, cudaStream_t stream);

// Accepted lengths and next tokens of sampled drafts, and the next step's pages (arguments already
// validated on the host; n_tok: rows, for uniform input too).
cudaError_t launch_sample(const gdn_sample &g, long long n_tok, int32_t *accepted, int32_t *next_ids,
                          cudaStream_t stream);
cudaError_t launch_pages(const gdn_pages &g, cudaStream_t stream);

// Linear attention (arguments already validated on the host); mode: kVerify, kCommit, or kFused
// for a step.
cudaError_t launch_linear(const LinearArgs &a, int mode, cudaStream_t stream);
// Rows a request from which the prompts' kernel runs: one number, although the three calls cross at other
// counts (left as it is).  64 requests of 32 heads of 128 x 128, all rows kept, us in the prompts' kernel / in the
// other: verify 182 / 125 at 47 rows, 186 / 330 at 64; step 205 / 180 at 24, 203 / 217 at 32; commit 193 / 125 at
// 47, 193 / 158 at 64.
constexpr int kLinearTcRows = 48;
bool linear_tc_runs(const gdn_linear &g);
cudaError_t launch_linear_tc(const LinearArgs &a, int mode, cudaStream_t stream);
bool linear_drafts_runs(const gdn_linear &g);  // a verify
cudaError_t launch_linear_drafts(const LinearArgs &a, cudaStream_t stream);

// One block that waits on a barrier nothing completes, until the bounded wait
// gives up; ORs GDN_DEVERR_TIMEOUT into *dev_err (not NULL).
cudaError_t launch_wait_selftest(int32_t *dev_err, cudaStream_t stream);

// Rotary positions and append (arguments already validated on the host; a.n_tok
// is the number of rows for uniform input too, a.o the rotated queries).
cudaError_t launch_rope(const AttnArgs &a, const gdn_rope &rope, bool bf16, const void *k,
                        long long k_stride, const void *v, long long v_stride, void *k_pages,
                        void *v_pages, cudaStream_t stream);

// Shared memory above 48 KB is asked for once a device and kernel (KERNEL names the
// instantiation, so each has its own record).
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};  // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// Chunk attention over the cache.  a.desc, a.count and a.part point into the workspace of
// attn_workspace() bytes: the descriptors, the counts, then the partials.
constexpr int kAttnWorkers = 304;    // blocks, two on each of 152 SMs
constexpr int kAttnHeader = 16384;   // bytes of the workspace before the partials
constexpr int kAttnLevels = 3;       // of counters
constexpr int kAttnTcWorkers = 152;  // one an SM: the tcgen05 kernel on prompt chunks
enum AttnKind { kAttnSimple, kAttnRows, kAttnDrafts, kAttnWide };
AttnKind attn_kind(bool bf16, int hd, long long rows);  // rows: max_T times the group
int64_t attn_workspace(bool bf16, int hd, long long rows);
cudaError_t launch_attn(AttnArgs a, bool bf16, cudaStream_t stream);
// Of launch_attn, the launch of one kernel, without that of combine_kernel.
cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_attn_tc(const AttnArgs &a, bool wide, cudaStream_t stream);

}  // namespace gdn
