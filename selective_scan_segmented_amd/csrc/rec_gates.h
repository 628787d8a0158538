// rec_gates.h -- the gates of the gated linear recurrence for one token and channel (gfx950).
//
//     la = -c softplus(lam) sigmoid(r),  a = exp(la),  m = sqrt(1 - a^2)
//
// The decay is kept as its base-2 logarithm, so that a is one exponential.  1 - a^2 = -expm1(2 la) cancels where a is
// near 1, which is where the recurrence remembers and where training starts (a from 0.9 to 0.999): there it is the
// series of expm1, elsewhere 1 - a a.
#pragma once

#include "sfm_device.h"

namespace sfm {

// sigmoid with the hardware's exponential and reciprocal (1 ulp each).  EXACT: the rounding of the exponent's
// product, which grows with |v|, is taken back to first order.
template <bool EXACT>
__device__ __forceinline__ float rec_sigmoid(float v) {
    float e;
    if constexpr (EXACT) {
        const float t = -v * kLog2e;
        const float err = __builtin_fmaf(-v, kLog2e, -t);
        e = exp2_fast(t);
        const float f = __builtin_fmaf(e, err * kLn2, e);
        e = __builtin_fabsf(v) < 80.0f ? f : e;  // (past that e overflows, or no longer counts beside 1)
    } else {
        e = exp2_fast(-v * kLog2e);
    }
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// -c softplus(lam) log2(e), a channel's constant; finite, so that a shut gate keeps the state at any rate.
__device__ __forceinline__ float rec_rate(float lam, float c) {
    const float rate = -c * softplus_log2e(lam);
    return rate < -3e38f ? -3e38f : rate;
}

// 1 - a^2 from la2 = log2(a) <= 0 and a itself.  The series' first omitted term and the rounding of 1 - a a meet at
// the threshold: EXACT (float32 tensors) z = 2 la > -1/2, eight terms, 2^-26 and 2^-22; else z > -1/16, four terms,
// 2^-23 and 2^-19.6, both of which the root halves.
template <bool EXACT>
__device__ __forceinline__ float rec_keep2(float la2, float a) {
    const float z = la2 * (2.0f * kLn2);
    float s;
    if constexpr (EXACT) {
        s = __builtin_fmaf(z, 1.0f / 8, 1.0f);
        s = __builtin_fmaf(z * (1.0f / 7), s, 1.0f);
        s = __builtin_fmaf(z * (1.0f / 6), s, 1.0f);
        s = __builtin_fmaf(z * (1.0f / 5), s, 1.0f);
        s = __builtin_fmaf(z * 0.25f, s, 1.0f);
    } else {
        s = __builtin_fmaf(z, 0.25f, 1.0f);
    }
    s = __builtin_fmaf(z * (1.0f / 3), s, 1.0f);
    s = __builtin_fmaf(z * 0.5f, s, 1.0f);
    s *= -z;
    return z > (EXACT ? -0.5f : -0.0625f) ? s : __builtin_fmaf(-a, a, 1.0f);
}

}  // namespace sfm
