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
    // workspace (backward with weights): [2][parts][d]
    float* part;
    int parts;
};

int64_t plan_rope_bwd(RopeParams& p, bool want);
hipError_t launch_rope_fwd(const RopeParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rope_bwd(const RopeParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
