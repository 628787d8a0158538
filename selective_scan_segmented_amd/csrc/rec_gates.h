// rec_gates.h -- the gates of the gated linear recurrence for one token and channel (gfx950).
//
//     la = -c softplus(lam) sigmoid(r),  a = exp(la),  m = sqrt(1 - a^2)
//
// The decay is kept as its base-2 logarithm, so that a is one exponential.  The difference 1 - a^2 cancels where a is
// near 1, which is where the recurrence remembers and where training starts (a from 0.9 to 0.999): there it is a series
// of sinh (rec_keep2), elsewhere 1 - a a.
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

// 1 - a^2 from la2 = log2(a) <= 0 and a itself: a (1/a - a) = 2 a sinh(w), w = -la2 ln 2, by the series of sinh, or 1 - a a.
// The series' first omitted term and an ulp of a in 1 - a a meet at the threshold.  What they leave in the root: EXACT
// (float32 tensors), w = 1/4, three terms: 2^-25 and 2^-22.4; else w = 1/16, two terms: 2^-24 and 2^-20.4.
template <bool EXACT>
__device__ __forceinline__ float rec_keep2(float la2, float a) {
    constexpr double w = 0.69314718055994531;  // ln 2
    constexpr double w3 = w * w * w;
    const float q = la2 * la2;
    float s = (float)(-w3 / 3);
    if constexpr (EXACT) s = __builtin_fmaf(q, (float)(-w3 * w * w / 60), s);
    s = __builtin_fmaf(q, s, (float)(-2 * w));
    float series = la2 * a * s, direct = __builtin_fmaf(-a, a, 1.0f);
    asm("" : "+v"(series), "+v"(direct));  // (both are made: a choice of lanes, not a branch for each value)
    return la2 > (float)((EXACT ? -0.25 : -0.0625) / w) ? series : direct;
}

}  // namespace sfm
