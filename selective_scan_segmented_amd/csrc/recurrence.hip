// recurrence.hip -- the gated linear recurrence (gfx950): forward, backward and one token of many requests.
//
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// and with G_t = dy_t + a_{t+1} G_{t+1}, s = sigmoid, m = sqrt(1 - a^2), P = G la (a h_{t-1} - a^2 / m s(i) x):
//
//     dx = G m s(i),  di = dx x (1 - s(i)),  dr = P (1 - s(r)),  dlam = s(lam) / softplus(lam) sum P,  dh0 = a_0 G_0.
//
// A lane walks one channel of a row token by token.
#include "rec_gates.h"
#include "sfm_rec.h"

namespace sfm {

namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void rec_fwd_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    const int d = blockIdx.y * kThreads + threadIdx.x, s = blockIdx.x;
    if (d >= p.D) return;
    int64_t first;
    int len;
    rec_row(p, s, first, len);
    const float rate = rec_rate(p.lam[d], p.c);
    float h = p.h0 ? p.h0[(int64_t)s * p.D + d] : 0.0f;
    const T* x = static_cast<const T*>(p.x) + first * p.ldx + d;
    const T* r = static_cast<const T*>(p.r) + first * p.ldr + d;
    const T* i = static_cast<const T*>(p.i) + first * p.ldi + d;
    T* y = static_cast<T*>(p.y) + first * p.D + d;
    for (int t = 0; t < len; ++t, x += p.ldx, r += p.ldr, i += p.ldi, y += p.D) {
        const float la2 = rate * rec_sigmoid<kExact>(to_f32(*r));
        const float a = exp2_fast(la2);
        const float m = __builtin_amdgcn_sqrtf(rec_keep2<kExact>(la2, a));
        h = __builtin_fmaf(a, h, m * rec_sigmoid<kExact>(to_f32(*i)) * to_f32(*x));
        *y = from_f32<T>(h);
    }
    if (p.hT) p.hT[(int64_t)s * p.D + d] = h;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rec_bwd_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    const int d = blockIdx.y * kThreads + threadIdx.x, s = blockIdx.x;
    if (d >= p.D) return;
    int64_t first;
    int len;
    rec_row(p, s, first, len);
    const float rate = rec_rate(p.lam[d], p.c);
    const float h0 = p.h0 ? p.h0[(int64_t)s * p.D + d] : 0.0f;
    float u = p.dhT ? p.dhT[(int64_t)s * p.D + d] : 0.0f, sum = 0.0f;
    for (int t = len - 1; t >= 0; --t) {
        const int64_t tok = first + t, at = tok * p.D + d;
        const float sr = rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.r)[tok * p.ldr + d]));
        const float si = rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.i)[tok * p.ldi + d]));
        const float x = to_f32(static_cast<const T*>(p.x)[tok * p.ldx + d]);
        const float before = t ? to_f32(static_cast<const T*>(p.y)[at - p.D]) : h0;
        const float la2 = rate * sr, a = exp2_fast(la2), em = rec_keep2<kExact>(la2, a);
        const float rs = em > 0.0f ? __builtin_amdgcn_rsqf(em) : 0.0f;
        const float G = to_f32(static_cast<const T*>(p.dy)[at]) + u;
        const float dx = G * (em * rs) * si;
        const float la = la2 * kLn2;
        const float P = G * (a * la) * (before - a * rs * si * x);
        sum += P;
        static_cast<T*>(p.dx)[at] = from_f32<T>(dx);
        static_cast<T*>(p.di)[at] = from_f32<T>(dx * x * (1.0f - si));
        static_cast<T*>(p.dr)[at] = from_f32<T>(P * (1.0f - sr));
        u = a * G;
    }
    if (p.dh0) p.dh0[(int64_t)s * p.D + d] = u;
    p.w_lam[(int64_t)s * p.D + d] = sum;
}

// dlam from the rows' parts.  softplus(lam) -> sigmoid(lam) (1 + e^lam / 2) as lam falls: their quotient is 1 in
// float32 below -17.
__global__ __launch_bounds__(64) void rec_lam_kernel(const RecParams p) {
    const int d = blockIdx.x * 64 + threadIdx.x;
    if (d >= p.D) return;
    float sum = 0.0f;
    for (int s = 0; s < p.rows; ++s) sum += p.w_lam[(int64_t)s * p.D + d];
    const float lam = p.lam[d];
    const float ratio = lam < -17.0f ? 1.0f : rec_sigmoid<true>(lam) / (softplus_log2e(lam) * kLn2);
    p.dlam[d] = sum * ratio;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void rec_step_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    const int d = blockIdx.y * kThreads + threadIdx.x, s = blockIdx.x;
    if (d >= p.D) return;
    const int64_t slot = p.slots ? p.slots[s] : s;
    T* y = static_cast<T*>(p.y) + (int64_t)s * p.D + d;
    if (slot < 0 || slot >= p.pool) {
        *y = from_f32<T>(0.0f);
        return;
    }
    float* state = p.hT + slot * p.D + d;
    const float la2 = rec_rate(p.lam[d], p.c) * rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.r)[s * p.ldr + d]));
    const float a = exp2_fast(la2), m = __builtin_amdgcn_sqrtf(rec_keep2<kExact>(la2, a));
    const float b = m * rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.i)[s * p.ldi + d])) *
                    to_f32(static_cast<const T*>(p.x)[s * p.ldx + d]);
    const float h = __builtin_fmaf(a, *state, b);
    *state = h;
    *y = from_f32<T>(h);
}

dim3 grid_of(const RecParams& p) { return dim3((unsigned)p.rows, (unsigned)((p.D + kThreads - 1) / kThreads)); }

}  // namespace

int64_t plan_rec_fwd(int64_t, int64_t, int64_t, int64_t, int) { return 0; }
int64_t plan_rec_bwd(int64_t rows, int64_t, int64_t, int64_t D, int) { return rows * D * 4; }

hipError_t launch_rec_fwd(const RecParams& p, int io_dtype, hipStream_t s) {
    if (io_dtype == 0)
        hipLaunchKernelGGL(rec_fwd_kernel<float>, grid_of(p), dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL(rec_fwd_kernel<__bf16>, grid_of(p), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_rec_bwd(const RecParams& p, int io_dtype, hipStream_t s) {
    if (io_dtype == 0)
        hipLaunchKernelGGL(rec_bwd_kernel<float>, grid_of(p), dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL(rec_bwd_kernel<__bf16>, grid_of(p), dim3(kThreads), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(rec_lam_kernel, dim3((unsigned)((p.D + 63) / 64)), dim3(64), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_rec_step(const RecParams& p, int io_dtype, hipStream_t s) {
    if (io_dtype == 0)
        hipLaunchKernelGGL(rec_step_kernel<float>, grid_of(p), dim3(kThreads), 0, s, p);
    else
        hipLaunchKernelGGL(rec_step_kernel<__bf16>, grid_of(p), dim3(kThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
