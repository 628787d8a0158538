// qk_rope.hip -- norm of every head's query and key with the position rotation in the same pass (gfx950).
//
//     xh = x / sqrt(mean x^2 + eps),  z = w xh,  (y1, y2) = (z1 cos - z2 sin, z2 cos + z1 sin)   angle = position * frequency
//
// for the pairs of the first `rot` values of a head, and with g the rotation back of dy
//
//     dw = sum of g xh,   dx = (w g - xh mean(w g xh)) / sqrt(mean x^2 + eps).
//
// A wave takes a head of a token, a lane its pairs lane and lane + 64.
#include "sfm_device.h"
#include "sfm_rope.h"

namespace sfm {

namespace {

constexpr int kWaves = 4;
constexpr int kMaxGroups = 2048;  // workgroups of a launch, each a strided part of the heads
constexpr float kRopeDown = 0x1p-96f;
constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)

// cos and sin of position * frequency: the product in turns and in 64 bits, its fraction to 32.
__device__ __forceinline__ void rope_angle(const RopeParams& p, int64_t tok, int j, float& c, float& s) {
    int axis = 0;
    for (int a = 0; a + 1 < p.axes; ++a) axis += j >= p.ends[a];
    const double turns = (double)p.positions[tok % p.period * p.axes + axis] * ((double)p.freqs[j] * kTurn);
    const double f = turns - __builtin_rint(turns);
    sincospif((float)(2.0 * f), &s, &c);
}

// The two values' places of pair slot j of a head: rotated pairs first, then the rest two by two (the last may be one).
__device__ __forceinline__ void rope_places(const RopeParams& p, int j, int& one, int& two) {
    const int half = p.rot >> 1;
    if (j < half && !p.neighbours) {
        one = j, two = j + half;
    } else {
        one = 2 * j, two = 2 * j + 1;
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

template <typename T, bool BACK>
__global__ __launch_bounds__(kWaves * 64) void rope_kernel(const RopeParams p) {
    __shared__ float red[kWaves][kRopeMaxD];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sd = blockIdx.y;
    const RopeSide q = p.side[sd];
    const int64_t heads = p.tokens * q.heads;
    float sums[4] = {0, 0, 0, 0};
    for (int64_t n = (int64_t)blockIdx.x * kWaves + wave; n < heads; n += (int64_t)gridDim.x * kWaves) {
        const int64_t tok = n / q.heads;
        const int h = (int)(n - tok * q.heads);
        const T* x = static_cast<const T*>(q.x) + tok * q.ld + (int64_t)h * p.d;
        float v[4] = {0, 0, 0, 0}, g[4] = {0, 0, 0, 0}, w[4] = {1, 1, 1, 1};
        int at[4];
        float sq = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            rope_places(p, lane + 64 * k, at[2 * k], at[2 * k + 1]);
#pragma unroll
            for (int m = 2 * k; m < 2 * k + 2; ++m)
                if (at[m] < p.d) {
                    v[m] = to_f32(x[at[m]]);
                    if (q.w) w[m] = q.w[at[m]];
                    if constexpr (BACK) g[m] = to_f32(static_cast<const T*>(q.dy)[n * p.d + at[m]]);
                    sq += v[m] * v[m];
                }
        }
        float rstd = 1.0f;
        if (p.norm) {
            sq = wave_sum(sq);
            float pre = 1.0f;
            if (__builtin_isinf(sq)) {  // squares past float32: the values' own scale first (eps is nothing beside them)
                pre = kRopeDown;
                sq = 0.0f;
#pragma unroll
                for (int m = 0; m < 4; ++m) v[m] *= pre, sq += v[m] * v[m];
                sq = wave_sum(sq);
            }
            rstd = 1.0f / __builtin_sqrtf(sq / (float)p.d + p.eps * pre * pre);
#pragma unroll
            for (int m = 0; m < 4; ++m) v[m] *= rstd;
            rstd *= pre;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float c = 1.0f, s = 0.0f;
            if (lane + 64 * k < p.rot >> 1) rope_angle(p, tok, lane + 64 * k, c, s);
            float& v1 = v[2 * k], & v2 = v[2 * k + 1], & g1 = g[2 * k], & g2 = g[2 * k + 1];
            if constexpr (BACK) {
                const float b1 = g1 * c + g2 * s, b2 = g2 * c - g1 * s;
                sums[2 * k] += b1 * v1, sums[2 * k + 1] += b2 * v2;
                g1 = b1 * w[2 * k], g2 = b2 * w[2 * k + 1];
            } else {
                const float z1 = v1 * w[2 * k], z2 = v2 * w[2 * k + 1];
                v1 = z1 * c - z2 * s, v2 = z2 * c + z1 * s;
            }
        }
        if constexpr (BACK) {
            float dot = 0.0f;
            if (p.norm) dot = wave_sum((g[0] * v[0] + g[1] * v[1]) + (g[2] * v[2] + g[3] * v[3])) / (float)p.d;
#pragma unroll
            for (int m = 0; m < 4; ++m) v[m] = rstd * (g[m] - v[m] * dot);
            // one value: 1 - xh^2 is eps / (x^2 + eps), of which the difference would leave nothing
            if (p.norm && p.d == 1) v[0] = rstd * g[0] * (p.eps * rstd * rstd);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m)
            if (at[m] < p.d) static_cast<T*>(q.y)[n * p.d + at[m]] = from_f32<T>(v[m]);
    }
    if constexpr (BACK) {
        if (!p.part) return;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            int at[2];
            rope_places(p, lane + 64 * k, at[0], at[1]);
            for (int m = 0; m < 2; ++m)
                if (at[m] < p.d) red[wave][at[m]] = sums[2 * k + m];
        }
        __syncthreads();
        for (int j = threadIdx.x; j < p.d; j += kWaves * 64) {
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < kWaves; ++m) sum += red[m][j];
            p.part[((int64_t)sd * p.parts + blockIdx.x) * p.d + j] = sum;
        }
    }
}

__global__ __launch_bounds__(64) void rope_weights_kernel(const RopeParams p) {
    const int j = blockIdx.x * 64 + threadIdx.x, sd = blockIdx.y;
    if (j >= p.d || !p.side[sd].dw) return;
    float sum = 0.0f;
    for (int m = 0; m < p.parts; ++m) sum += p.part[((int64_t)sd * p.parts + m) * p.d + j];
    p.side[sd].dw[j] = sum;
}

int groups_of(const RopeParams& p) {
    const int most = p.side[0].heads > p.side[1].heads ? p.side[0].heads : p.side[1].heads;
    const int64_t need = (p.tokens * most + kWaves - 1) / kWaves;
    return (int)(need < 1 ? 1 : need < kMaxGroups ? need : kMaxGroups);
}

}  // namespace

int64_t plan_rope_bwd(RopeParams& p, bool want) {
    p.parts = groups_of(p);
    return want ? 2 * (int64_t)p.parts * p.d * 4 : 0;
}

hipError_t launch_rope_fwd(const RopeParams& p, int io_dtype, hipStream_t s) {
    const dim3 grid(groups_of(p), 2);
    if (io_dtype == 0)
        hipLaunchKernelGGL((rope_kernel<float, false>), grid, dim3(kWaves * 64), 0, s, p);
    else
        hipLaunchKernelGGL((rope_kernel<__bf16, false>), grid, dim3(kWaves * 64), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_rope_bwd(const RopeParams& p, int io_dtype, hipStream_t s) {
    const dim3 grid(p.parts, 2);
    if (io_dtype == 0)
        hipLaunchKernelGGL((rope_kernel<float, true>), grid, dim3(kWaves * 64), 0, s, p);
    else
        hipLaunchKernelGGL((rope_kernel<__bf16, true>), grid, dim3(kWaves * 64), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.part) return e;
    hipLaunchKernelGGL(rope_weights_kernel, dim3((unsigned)((p.d + 63) / 64), 2), dim3(64), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
