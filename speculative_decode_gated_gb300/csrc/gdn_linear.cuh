// Shared pieces of the linear attention kernels (gdn_linear_*): the argument block, and a
// unit's rows and state with the device-side argument checks.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdn_device.cuh"

namespace gdn {

struct LinearArgs {
    gdn_linear g;              // n_tok is the number of rows for uniform input too
    int group;                 // heads that share a key head
    const int32_t *accepted;   // commit only, else NULL
    void *o;                   // NULL for commit
};

struct LinearUnit {
    int row0, T;               // rows to run (a commit's are the accepted ones)
    float *tile;               // the state, dk x dv
};

// A unit from its request's words, for calls without accepted lengths; report: this thread reports what
// is wrong with it.  False: skip the unit.
__device__ __forceinline__ bool linear_words(const LinearArgs &a, long long c0, long long c1, int slot, int h,
                                             LinearUnit &u, bool report) {
    const gdn_linear &g = a.g;
    int err = 0;
    const long long T = c1 - c0;
    if (T < 0 || T > g.max_T || c0 < 0 || c1 > g.n_tok) err |= GDN_DEVERR_SEQLEN;
    if (slot < 0 || slot >= g.pool_slots) err |= GDN_DEVERR_SLOT;
    if (err) {
        if (report && g.dev_err) atomicOr(g.dev_err, err);
        return false;
    }
    u.row0 = (int)c0;
    u.T = (int)T;
    u.tile = g.pool + ((long long)slot * g.heads + h) * ((long long)g.dk * g.dv);
    return T > 0;
}

// Every thread of the block calls it and finds the same answer; thread 0 reports.  commit: T is the accepted length.
__device__ __forceinline__ bool linear_unit(const LinearArgs &a, int r, int h, bool commit, LinearUnit &u) {
    const gdn_linear &g = a.g;
    long long c0 = (long long)r * g.max_T, c1 = c0 + g.max_T;
    if (g.cu_seqlens) {
        c0 = g.cu_seqlens[r];
        c1 = g.cu_seqlens[r + 1];
    }
    const int slot = g.slot_ids[r];
    const int acc = commit ? a.accepted[r] : 0;
    LinearUnit x;
    x.T = 0;
    const bool rows = linear_words(a, c0, c1, slot, h, x, threadIdx.x == 0);
    if (!commit) {
        if (rows) u = x;
        return rows;
    }
    if (acc < 0 || acc > (rows ? x.T : 0)) {
        // (of a request that is skipped already, nothing more is reported)
        const bool good = rows || (c1 == c0 && c0 >= 0 && c1 <= g.n_tok && slot >= 0 && slot < g.pool_slots);
        if (good && threadIdx.x == 0 && g.dev_err) atomicOr(g.dev_err, GDN_DEVERR_ACCEPTED);
        return false;
    }
    if (!rows) return false;
    u = x;
    u.T = acc;
    return acc > 0;
}

}  // namespace gdn
