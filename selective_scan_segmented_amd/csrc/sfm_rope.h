// sfm_rope.h -- host/device contract of the norm and rotation of queries and keys (qk_rope.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfm {

constexpr int kRopeMaxD = 256;   // largest head
constexpr int kRopeMaxAxes = 4;  // position axes

// queries (0) and keys (1) of a call
struct RopeSide {
    const void* x;    // token t, head h: x + t * ld + h * d (elements)
    const void* dy;   // backward: [tokens][heads][d]
    const float* w;   // [d] or null (1)
    void* y;          // [tokens][heads][d]; backward: dx
    float* dw;        // backward: [d] or null (not wanted)
    int64_t ld;
    int heads;
    int run;          // tokens that a workgroup takes at a time
    int64_t groups;   // workgroups; backward: no more than kRopeParts
};

struct RopeParams {
    RopeSide side[2];
    const int32_t* positions;  // [period][axes]: token t has row t % period
    const float* freqs;        // [rot / 2]: angle = position * frequency
    int64_t tokens, period;
    int d, rot, axes;          // rot 0: no rotation
    int ends[kRopeMaxAxes];    // pair j goes by the first axis a with j < ends[a]
    float eps;
    int norm, neighbours;      // neighbours: pairs (2j, 2j + 1), else (j, j + rot / 2)
    // plan (plan_rope)
    int vec;                   // neighbouring values to a load
    int slots, lanes;          // of two vec to a head; lanes: to a head, a power of two
    int threads;
    int lines;                 // outputs written past the cache
    float* part;               // workspace (backward with weights): [2][kRopeParts][d]
};

constexpr int kRopeParts = 1024;  // most parts of dw to a side

// Fills the plan; align: bytes that every tensor's rows are aligned to (16, 8, 4 or 2).
void plan_rope(RopeParams& p, int io_bytes, int align, bool back);
hipError_t launch_rope_fwd(const RopeParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rope_bwd(const RopeParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
