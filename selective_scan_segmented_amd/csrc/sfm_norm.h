// sfm_norm.h -- host/device contract of the channel-last group norm (group_norm.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfm {

struct NormParams {
    const void* x;       // [N][L][C]
    const void* dy;      // backward: [N][L][C]
    const float* w;      // [C] or null (1)
    const float* b;      // [C] or null (0)
    void* y;             // forward: output; backward: dx
    float* mean;         // [N][G]: written by the forward, read by the backward
    float* rstd;
    float* dw;           // [C] or null
    float* db;
    int64_t N, L;
    int C, G, cg;        // cg = C / G
    float eps;
    int act;
    // plan (plan_norm)
    int vec;             // channels to a unit of 16 bytes, or 1
    int slab;            // 1: a sample's run of whole groups stays in a workgroup's registers; 0: two passes
    int cw, runs;        // slab: channels to a run (whole groups), runs to a row
    int threads, units;  // workgroup size, units a thread holds (slab)
    int tiles, tunits;   // two passes: channel tiles to a row, units to a tile
    int splits;          // two passes: row ranges a sample
    int64_t srows;       // rows to a range
    float* part;         // workspace: per-channel sums [N][splits][2][C]
};

// Fills the plan; returns the workspace bytes of the call.
int64_t plan_norm(NormParams& p, int io_bytes, bool aligned, bool backward);
hipError_t launch_group_norm_fwd(const NormParams& p, int io_dtype, hipStream_t s);
hipError_t launch_group_norm_bwd(const NormParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
