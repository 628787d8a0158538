// sfm_rec.h -- host/device contract of the gated linear recurrence's kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfm {

// One call's rows, channels and strides (forward, backward and the step).
struct RecParams {
    const void* x;           // token t, channel d: x + t * ldx + d (elements)
    const void* r;
    const void* i;
    const float* lam;        // [D]
    const float* h0;         // [rows][D] or null (zero); the pool with the step
    void* y;                 // [tokens][D]; read by the backward
    float* hT;               // [rows][D] or null; the pool with the step
    const int32_t* offsets;  // [rows + 1] or null: row s is tokens s * L .. + L - 1
    const int32_t* slots;    // [rows] or null: the state of row s is number slots[s] of `pool`
    int64_t ldx, ldr, ldi, tokens, pool;
    int rows, L, D;
    float c;
    // backward
    const void* dy;          // [tokens][D]
    const float* dhT;        // [rows][D] or null (zero)
    void *dx, *dr, *di;      // [tokens][D]
    float* dlam;             // [D]
    float* dh0;              // [rows][D] or null
    float* w_lam;            // workspace: [rows][D], every row's part of dlam
};

// first token and length of row s; offsets outside the tokens (a caller's mistake) are cut to them
__device__ __forceinline__ void rec_row(const RecParams& p, int s, int64_t& first, int& len) {
    if (!p.offsets) {
        first = (int64_t)s * p.L;
        len = p.L;
        return;
    }
    int64_t lo = p.offsets[s], hi = p.offsets[s + 1];
    lo = lo < 0 ? 0 : (lo > p.tokens ? p.tokens : lo);
    hi = hi < lo ? lo : (hi > p.tokens ? p.tokens : hi);
    first = lo;
    len = hi - lo > p.L ? p.L : (int)(hi - lo);
}

// Workspace bytes of the calls.
int64_t plan_rec_fwd(int64_t rows, int64_t L, int64_t tokens, int64_t D, int io_dtype);
int64_t plan_rec_bwd(int64_t rows, int64_t L, int64_t tokens, int64_t D, int io_dtype);
hipError_t launch_rec_fwd(const RecParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rec_bwd(const RecParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rec_step(const RecParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
