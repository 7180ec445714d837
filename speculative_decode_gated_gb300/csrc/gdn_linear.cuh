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

// Every thread of the block finds the same answer; thread 0 reports.  False: skip the unit.
__device__ __forceinline__ bool linear_unit(const LinearArgs &a, int r, int h, bool commit, LinearUnit &u) {
    const gdn_linear &g = a.g;
    long long c0 = (long long)r * g.max_T, c1 = c0 + g.max_T;
    if (g.cu_seqlens) {
        c0 = g.cu_seqlens[r];
        c1 = g.cu_seqlens[r + 1];
    }
    const int slot = g.slot_ids[r];
    int err = 0;
    long long T = c1 - c0;
    if (T < 0 || T > g.max_T || c0 < 0 || c1 > g.n_tok) err |= GDN_DEVERR_SEQLEN;
    if (slot < 0 || slot >= g.pool_slots) err |= GDN_DEVERR_SLOT;
    if (commit) {
        const int acc = a.accepted[r];
        if (!err && (acc < 0 || acc > T)) err |= GDN_DEVERR_ACCEPTED;
        T = acc;
    }
    if (err) {
        if (threadIdx.x == 0 && g.dev_err) atomicOr(g.dev_err, err);
        return false;
    }
    u.row0 = (int)c0;
    u.T = (int)T;
    u.tile = g.pool + ((long long)slot * g.heads + h) * ((long long)g.dk * g.dv);
    return T > 0;
}

}  // namespace gdn
