// qk_rope.hip -- norm of every head's query and key with the position rotation in the same pass (gfx950).
//
//     xh = x / sqrt(mean x^2 + eps),  z = w xh,  (y1, y2) = (z1 cos - z2 sin, z2 cos + z1 sin)   angle = position * frequency
//
// for the pairs of the first `rot` values of a head, and with g the rotation back of dy
//
//     dw = sum of g xh,   dx = (w g - xh mean(w g xh)) / sqrt(mean x^2 + eps).
//
// Bound by memory: 4 bytes a bfloat16 value forward, 6 backward, and some 15 and 25 lane operations.  A head lies in a
// power of two of lanes, each with two runs of up to 16 bytes that hold both values of its pairs (the run and the one
// half a rotation on, or 2 x 16 bytes side by side), so that the rotation stays in a lane and the mean square is one sum
// over a few.  A workgroup takes a run of tokens with all heads of queries or of keys: it makes the tokens' sines and
// cosines once, into LDS, while its first heads are on their way.
// Measured, bfloat16: forward, 256 x 198 tokens x 10 heads of 64: 28 us, 4.6 TB/s; 2 x 8192 x 24 heads of 128: 38 us, 5.2
// TB/s; backward, 2 x 4002 x 12 heads of 128: 21 us, 3.5 TB/s, of which 4 are the weights' join (a copy of its 74 MB: 19).
// Calls back to back: 2 x 8192 x 24 heads of 128, backward 60 us, 5.0 TB/s; neighbours 43 us; float32 73 us, backward 120 us,
// neighbours 84 us.
#include "sfm_device.h"
#include "sfm_rope.h"

namespace sfm {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;  // sines and cosines that a workgroup holds
constexpr int kPositions = 512;  // and positions
constexpr float kRopeDown = 0x1p-96f;
constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)

// V neighbouring values as they lie in memory.
template <typename T, int V> struct RopeRun {
    static constexpr int kBytes = V * (int)sizeof(T), kWords = kBytes < 4 ? 1 : kBytes / 4;
    uint32_t w[kWords];
    typedef uint32_t w2 __attribute__((ext_vector_type(2)));
    typedef uint32_t w4 __attribute__((ext_vector_type(4)));
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t b, uint32_t at) {
        if constexpr (kBytes == 16) {
            const w4 v = __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = v[k];
        } else if constexpr (kBytes == 8) {
            const w2 v = __builtin_amdgcn_raw_buffer_load_b64(b, at, 0, 0);
            w[0] = v[0], w[1] = v[1];
        } else if constexpr (kBytes == 4) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0);
        } else {
            w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0);
        }
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
    }
    template <int POLICY>
    static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t b, uint32_t at, const float (&f)[V]) {
        uint32_t w[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (sizeof(T) == 4) {
                w[k] = __float_as_uint(f[k]);
            } else {
                typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
                w[k] = __builtin_bit_cast(uint32_t, bf2{(__bf16)f[2 * k], (__bf16)f[V > 1 ? 2 * k + 1 : 2 * k]});
            }
        }
        if constexpr (kBytes == 16)
            __builtin_amdgcn_raw_buffer_store_b128(w4{w[0], w[1], w[2], w[3]}, b, at, 0, POLICY);
        else if constexpr (kBytes == 8)
            __builtin_amdgcn_raw_buffer_store_b64(w2{w[0], w[1]}, b, at, 0, POLICY);
        else if constexpr (kBytes == 4)
            __builtin_amdgcn_raw_buffer_store_b32(w[0], b, at, 0, POLICY);
        else
            __builtin_amdgcn_raw_buffer_store_b16((unsigned short)w[0], b, at, 0, POLICY);
    }
};

// cos and sin of position * frequency: the product in turns and in 64 bits, its fraction to 32.  Beside bfloat16 values
// the hardware's functions of turns are exact enough (of sines and cosines alone, 1 in 10000 rounds to the neighbour of
// the exact value's); float32 ones take the library's.
template <bool EXACT>
__device__ __forceinline__ float2 rope_angle(int position, float freq) {
    const double turns = (double)position * ((double)freq * kTurn);
    const float f = (float)(turns - __builtin_rint(turns));
    float2 cs;
    if constexpr (EXACT)
        sincospif(2.0f * f, &cs.y, &cs.x);
    else
        cs = make_float2(__builtin_amdgcn_cosf(f), __builtin_amdgcn_sinf(f));
    return cs;
}

// Sum over a power of two of neighbouring lanes, in all of them.
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#define SFM_DPP(ctrl) v += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), ctrl, 0xf, 0xf, true))
    if (lanes > 1) SFM_DPP(0xb1);   // quad_perm 1, 0, 3, 2
    if (lanes > 2) SFM_DPP(0x4e);   // quad_perm 2, 3, 0, 1
    if (lanes > 4) SFM_DPP(0x141);  // row_half_mirror: the other quad of eight
    if (lanes > 8) SFM_DPP(0x140);  // row_mirror: the other eight of a row
#undef SFM_DPP
    if (lanes > 16) v += __shfl_xor(v, 16);
    if (lanes > 32) v += __shfl_xor(v, 32);
    return v;
}

// The pairs of a lane's two runs turned by (cos, sin): value v of one with that of the other, or neighbours in each.
template <int V, bool NEIGH>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2* cs, float sign) {
    auto pair = [&](float& x, float& y, float2 t) __attribute__((always_inline)) {
        const float s = sign * t.y, x1 = x * t.x - y * s;
        y = y * t.x + x * s;
        x = x1;
    };
    if constexpr (NEIGH && V > 1) {
#pragma unroll
        for (int m = 0; m < V / 2; ++m) {
            pair(a[2 * m], a[2 * m + 1], cs[m]);
            pair(b[2 * m], b[2 * m + 1], cs[V / 2 + m]);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) pair(a[v], b[v], cs[v]);
    }
}

// Heads that a lane has in flight: as many as registers allow (forward of 2 x 8192 tokens x 24 heads of 128: 40 us with
// four, 42 with two, 58 with one; backward of 2 x 4002 x 12: 23.2 us with one, 24 with two).
constexpr int in_flight(int V, int S, bool back) { return S > 1 || back ? 1 : 4; }

// S: slots to a lane.
template <typename T, int V, int S, bool NEIGH, bool BACK>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeParams p) {
    constexpr int U = in_flight(V, S, BACK);
    __shared__ __align__(16) float2 table[kTable];
    __shared__ int positions[kPositions];
    __shared__ float freqs[kRopeMaxD / 2];
    const int sd = blockIdx.y, tid = threadIdx.x;
    const RopeSide& q = p.side[sd];
    if ((int64_t)blockIdx.x >= q.groups) return;
    const int lane = tid & (p.lanes - 1), group = tid / p.lanes, groups = (int)blockDim.x / p.lanes;
    const int half = p.rot >> 1, width = p.slots * V;
    int one[S], two[S];
    bool pairs[S];  // the slot's values are rotated; others stay as they are, whatever stands beside them
    float w1[S][V], w2[S][V], s1[S][V], s2[S][V];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int slot = lane + 64 * s;
        one[s] = slot * V, two[s] = half + slot * V;
        pairs[s] = slot * V < half;
        if (NEIGH || !pairs[s]) one[s] = 2 * slot * V, two[s] = one[s] + V;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            w1[s][v] = q.w && one[s] < p.d ? q.w[one[s] + v] : 1.0f;
            w2[s][v] = q.w && two[s] < p.d ? q.w[two[s] + v] : 1.0f;
            s1[s][v] = s2[s][v] = 0.0f;
        }
    }
    const float inv_heads = 1.0f / (float)q.heads, inv_d = 1.0f / (float)p.d, inv_width = 1.0f / (float)width;
    const float inv_axes = 1.0f / (float)p.axes;
    if (tid < half) freqs[tid] = p.freqs[tid];
    const uint32_t period = (uint32_t)p.period;
    for (int64_t run = blockIdx.x; run * q.run < p.tokens; run += q.groups) {
        const int64_t tok0 = run * q.run;
        const int tokens = p.tokens - tok0 < q.run ? (int)(p.tokens - tok0) : q.run, rows = tokens * q.heads;
        const __amdgpu_buffer_rsrc_t xb = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(q.x) + tok0 * q.ld), 0, -1, 0x00027000);
        const int64_t out = tok0 * q.heads * p.d;
        const __amdgpu_buffer_rsrc_t yb = __builtin_amdgcn_make_buffer_rsrc(static_cast<T*>(q.y) + out, 0, -1, 0x00027000);
        const __amdgpu_buffer_rsrc_t gb = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(BACK ? q.dy : q.x) + (BACK ? out : 0)), 0, -1, 0x00027000);
        // the run's positions: asked for before its first heads, so that they are there first
        int at[kPositions / kThreads];
        const uint32_t base = (uint32_t)tok0 % period;  // (the same for all lanes)
#pragma unroll
        for (int e = 0; e < kPositions / kThreads; ++e) {
            at[e] = 0;
            const int k = tid + e * kThreads;
            if (!half || k >= tokens * p.axes) continue;
            const int t = div_small(k, inv_axes);
            uint32_t row = base + (uint32_t)t;
            if (row >= period) row = row - period < period ? row - period : row % period;
            at[e] = p.positions[(int64_t)row * p.axes + (k - t * p.axes)];
        }
        for (int r0 = 0; r0 < rows; r0 += groups * U) {
            RopeRun<T, V> x1[U][S], x2[U][S], g1[U][S], g2[U][S];
            int tok[U];
            uint32_t to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int row = r0 + u * groups + group;
                tok[u] = div_small(row, inv_heads);
                const int h = row - tok[u] * q.heads;
                to[u] = (uint32_t)row * p.d * sizeof(T);
                const uint32_t from = ((uint32_t)tok[u] * (uint32_t)q.ld + h * p.d) * sizeof(T);
#pragma unroll
                for (int s = 0; s < S; ++s)
                    if (row < rows) {
                        if (one[s] < p.d) {
                            x1[u][s].load(xb, from + one[s] * sizeof(T));
                            if constexpr (BACK) g1[u][s].load(gb, to[u] + one[s] * sizeof(T));
                        }
                        if (two[s] < p.d) {
                            x2[u][s].load(xb, from + two[s] * sizeof(T));
                            if constexpr (BACK) g2[u][s].load(gb, to[u] + two[s] * sizeof(T));
                        }
                    }
            }
            if (r0 == 0) {  // the run's sines and cosines (places of values behind the rotation are left empty)
#pragma unroll
                for (int e = 0; e < kPositions / kThreads; ++e) positions[tid + e * kThreads] = at[e];
                lds_barrier();
                for (int k = tid; k < tokens * width; k += kThreads) {
                    const int t = div_small(k, inv_width), j = k - t * width;
                    int axis = 0;
                    for (int a = 0; a + 1 < p.axes; ++a) axis += j >= p.ends[a];
                    if (j < half) table[k] = rope_angle<sizeof(T) == 4>(positions[t * p.axes + axis], freqs[j]);
                }
                lds_barrier();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool live = r0 + u * groups + group < rows;
                float a[S][V], b[S][V], sq = 0.0f;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        a[s][v] = live && one[s] < p.d ? x1[u][s].get(v) : 0.0f;
                        b[s][v] = live && two[s] < p.d ? x2[u][s].get(v) : 0.0f;
                        sq = __builtin_fmaf(a[s][v], a[s][v], sq);
                        sq = __builtin_fmaf(b[s][v], b[s][v], sq);
                    }
                float rstd = 1.0f;
                if (p.norm) {
                    sq = lanes_sum(sq, p.lanes);
                    float pre = 1.0f;
                    if (__any(__builtin_isinf(sq))) {  // squares past float32: the values' own scale first (eps is nothing beside them)
                        pre = __builtin_isinf(sq) ? kRopeDown : 1.0f;
                        sq = 0.0f;
#pragma unroll
                        for (int s = 0; s < S; ++s)
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                a[s][v] *= pre, b[s][v] *= pre;
                                sq = __builtin_fmaf(a[s][v], a[s][v], sq);
                                sq = __builtin_fmaf(b[s][v], b[s][v], sq);
                            }
                        sq = lanes_sum(sq, p.lanes);
                    }
                    rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(sq, inv_d, p.eps * pre * pre));
#pragma unroll
                    for (int s = 0; s < S; ++s)
#pragma unroll
                        for (int v = 0; v < V; ++v) a[s][v] *= rstd, b[s][v] *= rstd;
                    rstd *= pre;
                }
                const float2* cs = table + (live ? tok[u] : 0) * width;
                if constexpr (!BACK) {
#pragma unroll
                    for (int s = 0; s < S; ++s) {
#pragma unroll
                        for (int v = 0; v < V; ++v) a[s][v] *= w1[s][v], b[s][v] *= w2[s][v];
                        if (pairs[s]) turn<V, NEIGH>(a[s], b[s], cs + (lane + 64 * s) * V, 1.0f);
                    }
                } else {
                    float e[S][V], f[S][V], dot = 0.0f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            e[s][v] = live && one[s] < p.d ? g1[u][s].get(v) : 0.0f;
                            f[s][v] = live && two[s] < p.d ? g2[u][s].get(v) : 0.0f;
                        }
                        if (pairs[s]) turn<V, NEIGH>(e[s], f[s], cs + (lane + 64 * s) * V, -1.0f);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            s1[s][v] = __builtin_fmaf(e[s][v], a[s][v], s1[s][v]);
                            s2[s][v] = __builtin_fmaf(f[s][v], b[s][v], s2[s][v]);
                            e[s][v] *= w1[s][v], f[s][v] *= w2[s][v];
                            dot = __builtin_fmaf(e[s][v], a[s][v], dot);
                            dot = __builtin_fmaf(f[s][v], b[s][v], dot);
                        }
                    }
                    if (p.norm) {
                        dot = lanes_sum(dot, p.lanes) * inv_d;
#pragma unroll
                        for (int s = 0; s < S; ++s)
#pragma unroll
                            for (int v = 0; v < V; ++v) {
                                a[s][v] = rstd * __builtin_fmaf(-a[s][v], dot, e[s][v]);
                                b[s][v] = rstd * __builtin_fmaf(-b[s][v], dot, f[s][v]);
                            }
                        // one value: 1 - xh^2 is eps / (x^2 + eps), of which the difference would leave nothing
                        if (p.d == 1) a[0][0] = rstd * e[0][0] * (p.eps * rstd * rstd);
                    } else {
#pragma unroll
                        for (int s = 0; s < S; ++s)
#pragma unroll
                            for (int v = 0; v < V; ++v) a[s][v] = e[s][v], b[s][v] = f[s][v];
                    }
                }
                auto put = [&](auto policy) __attribute__((always_inline)) {
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        if (one[s] < p.d) RopeRun<T, V>::template store<decltype(policy)::value>(yb, to[u] + one[s] * sizeof(T), a[s]);
                        if (two[s] < p.d) RopeRun<T, V>::template store<decltype(policy)::value>(yb, to[u] + two[s] * sizeof(T), b[s]);
                    }
                };
                if (live) {
                    if (!BACK && !NEIGH && V > 1 && p.lines)
                        put(std::integral_constant<int, 2>{});  // (nontemporal)
                    else
                        put(std::integral_constant<int, 0>{});
                }
            }
        }
        lds_barrier();  // (the next run's table)
    }
    if constexpr (BACK) {
        if (!p.part) return;
        // the lanes of a wave with the same values, then the waves
        float* red = reinterpret_cast<float*>(table);  // [waves][kRopeMaxD]: 1024 of 4096 floats
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                for (int m = p.lanes; m < 64; m <<= 1) {
                    s1[s][v] += __shfl_xor(s1[s][v], m);
                    s2[s][v] += __shfl_xor(s2[s][v], m);
                }
                if ((tid & 63) < p.lanes) {
                    if (one[s] < p.d) red[(tid >> 6) * kRopeMaxD + one[s] + v] = s1[s][v];
                    if (two[s] < p.d) red[(tid >> 6) * kRopeMaxD + two[s] + v] = s2[s][v];
                }
            }
        lds_barrier();
        for (int j = tid; j < p.d; j += blockDim.x) {
            float sum = 0.0f;
            for (int m = 0; m < (int)blockDim.x / 64; ++m) sum += red[m * kRopeMaxD + j];
            p.part[((int64_t)sd * kRopeParts + blockIdx.x) * p.d + j] = sum;
        }
    }
}

// dw from the workgroups' parts: 16 values to a workgroup, every 64th part to a lane, all asked for together.
__global__ __launch_bounds__(1024) void rope_weights_kernel(const RopeParams p) {
    __shared__ float part[64][17];
    const int w = threadIdx.x & 15, g = threadIdx.x >> 4, j = blockIdx.x * 16 + w;
    const RopeSide& q = p.side[blockIdx.y];
    if (!q.dw) return;
    float sum = 0.0f;
    if (j < p.d) {
        const float* v = p.part + (int64_t)blockIdx.y * kRopeParts * p.d + j;
        const int n = (int)q.groups;
        float f[kRopeParts / 64];
#pragma unroll
        for (int m = 0; m < kRopeParts / 64; ++m) f[m] = m * 64 + g < n ? v[(m * 64 + g) * p.d] : 0.0f;
#pragma unroll
        for (int m = 0; m < kRopeParts / 64; ++m) sum += f[m];
    }
    part[g][w] = sum;
    lds_barrier();
    if (g >= 16) return;
    sum = ((part[g][w] + part[g + 16][w]) + part[g + 32][w]) + part[g + 48][w];
    part[g][w] = sum;  // (its own place, read by none but it before the barrier)
    lds_barrier();
    if (g || j >= p.d) return;
    for (int k = 1; k < 16; ++k) sum += part[k][w];
    q.dw[j] = sum;
}

template <typename T, bool NEIGH, bool BACK>
hipError_t launch_t(const RopeParams& p, hipStream_t s) {
    const int64_t most = p.side[0].groups > p.side[1].groups ? p.side[0].groups : p.side[1].groups;
    const dim3 grid((unsigned)most, 2), threads(p.threads);
#define SFM_ROPE(V, S) hipLaunchKernelGGL((rope_kernel<T, V, S, NEIGH, BACK>), grid, threads, 0, s, p)
    constexpr int W = 16 / (int)sizeof(T);  // (the backward: 8 bytes at most, plan_rope)
    if (p.vec == W) {
        if constexpr (!BACK) SFM_ROPE(W, 1);
    } else if (p.vec == 4) {
        if constexpr (W == 8) SFM_ROPE(4, 1);
    } else if (p.vec == 2) {
        SFM_ROPE(2, 1);
    } else if (p.slots <= 64) {
        SFM_ROPE(1, 1);
    } else {
        SFM_ROPE(1, 2);
    }
#undef SFM_ROPE
    return hipGetLastError();
}

template <bool BACK>
hipError_t launch(const RopeParams& p, int io_dtype, hipStream_t s) {
    if (io_dtype == 0) return p.neighbours ? launch_t<float, true, BACK>(p, s) : launch_t<float, false, BACK>(p, s);
    return p.neighbours ? launch_t<__bf16, true, BACK>(p, s) : launch_t<__bf16, false, BACK>(p, s);
}

}  // namespace

void plan_rope(RopeParams& p, int io_bytes, int align, bool back) {
    // The widest run that both parts of a head, its tokens' strides and its tensors' alignment are whole pairs of, up to
    // 16 bytes; of the backward 8, which leaves more waves registers (2 x 4002 tokens x 12 heads of 128: 24.6 us, 27.2
    // with 16, at two heads in flight 32.5).
    int V = (back ? 8 : 16) / io_bytes;
    const int rest = p.d - p.rot;
    while (V > 1 && (p.rot % (2 * V) || rest % (2 * V) || p.side[0].ld % V || p.side[1].ld % V || align < V * io_bytes)) V /= 2;
    p.vec = V;
    p.slots = (p.d + 2 * V - 1) / (2 * V);
    p.lanes = 1;
    while (p.lanes < p.slots && p.lanes < 64) p.lanes *= 2;
    const int per = in_flight(V, p.slots > 64 ? 2 : 1, back) * (back ? 8 : 1);
    p.threads = kThreads;
    // Outputs whose halves are whole lines of 128 bytes are written past the cache (without / with it: 2 x 8192 tokens x 24 heads
    // of 128 among other work: 44 / 38 us, between a writer of q and k and a reader of both outputs 113 / 112 us).  Not others:
    // 256 x 198 x 10 heads of 64, so placed: 75 / 80 us; nor the backward, 8 x 8192 x 24 heads of 128: 526 / 538 us.
    p.lines = !back && !p.neighbours && p.rot == p.d && p.d / 2 * io_bytes % 128 == 0;
    for (RopeSide& q : p.side) {
        // tokens whose heads give every lane that many, as far as the table holds them and enough workgroups are left
        int64_t run = (int64_t)(kThreads / p.lanes) * per / q.heads;
        const int64_t of_table = kTable / (p.slots * V), of_positions = kPositions / p.axes;
        const int64_t holds = of_table < of_positions ? of_table : of_positions, few = p.tokens / 512;
        if (run > holds) run = holds;
        if (run > few) run = few;
        const int64_t near = (1LL << 31) / (q.ld * io_bytes);  // (whose bytes stay below 2^31)
        if (run > near) run = near;
        q.run = run < 1 ? 1 : (int)run;
        q.groups = (p.tokens + q.run - 1) / q.run;
        const int64_t most = back ? kRopeParts : 1 << 20;  // (a launch holds fewer than 2^32 work items)
        if (q.groups > most) q.groups = most;
    }
}

hipError_t launch_rope_fwd(const RopeParams& p, int io_dtype, hipStream_t s) { return launch<false>(p, io_dtype, s); }

hipError_t launch_rope_bwd(const RopeParams& p, int io_dtype, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (p.tokens > 0) e = launch<true>(p, io_dtype, s);
    if (e != hipSuccess || !p.part) return e;
    hipLaunchKernelGGL(rope_weights_kernel, dim3((unsigned)((p.d + 15) / 16), 2), dim3(1024), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
