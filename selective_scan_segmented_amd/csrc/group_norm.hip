// group_norm.hip -- group norm of channel-last tokens with an optional SiLU, forward and backward (gfx950).
//
//     mean, var over the L x C/G values of a sample's group;  xh = (x - mean) / sqrt(var + eps);
//     z = w xh + b;  y = z or z sigmoid(z)
//     backward: dz = dy act'(z);  db = sum dz;  dw = sum dz xh;
//               dx = rstd (w dz - m1 - xh m2),  m1, m2 the group's means of w dz and w dz xh
//
// Bound by memory: x and y once (forward), x, dy and dx once (backward), against some ten operations a value.  A
// thread owns one 16-byte unit of channels and walks down rows, so loads are whole cache lines whatever the group
// width, and both directions need per-channel sums only; a group's are the sums of its channels'.
//
// * Slab kernels: a sample's rows of some whole groups stay in the registers of one workgroup from the load to the
//   store (one read, one write, one launch).  The mean is taken first and the squares about it, so a mean far from
//   zero costs no digits.
// * Two passes, where a group does not fit: row ranges of a sample to separate workgroups, which leave per-channel
//   sums; a small kernel joins them in a fixed order; the second pass reads the input again (from the last-level
//   cache if it fits there).  Squares are taken about the mean of each batch of eight rows, and batches, channels
//   and ranges are joined by the exact formula for the squares of a union, again so that a large mean costs nothing.
// Sums are float32 in a fixed order: repeated calls give the same bits.
#include "sfm_device.h"
#include "sfm_norm.h"

namespace sfm {

namespace {

template <typename T, int V> struct alignas(V * sizeof(T)) Unit {
    T e[V];
};

// sigmoid without overflow: exp2 of a large positive argument is infinity and 1 / infinity is 0
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + exp2_fast(-z * kLog2e)); }

__device__ __forceinline__ float act_fwd(float z, int act) { return act ? z * sigmoid(z) : z; }

// dy act'(z)
__device__ __forceinline__ float act_bwd(float dy, float z, int act) {
    if (!act) return dy;
    const float s = sigmoid(z);
    return dy * (s * __builtin_fmaf(z, 1.0f - s, 1.0f));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Sum of each group's entries of buf [slots][cw] into out[groups of the run]: a wave to a group.
__device__ __forceinline__ void group_sums(const float* buf, int slots, int cw, int cg, float* out) {
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    for (int g = threadIdx.x >> 6; g < cw / cg; g += waves) {
        float v = 0.0f;
        const int n = slots * cg;
        for (int i = lane; i < n; i += 64) {
            const int s = i / cg;
            v += buf[s * cw + g * cg + (i - s * cg)];
        }
        v = wave_sum(v);
        if (lane == 0) out[g] = v;
    }
}

// ------------------------------------------------------------------------------------------------ slab kernels
// LDS: [slots][cw] per-thread channel sums (two of them backward), then the groups' sums.
template <typename T, int V, int U>
__global__ __launch_bounds__(1024) void norm_slab_fwd_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const int cu = p.cw / V, slots = blockDim.x / cu;
    const int64_t n = blockIdx.x / p.runs;
    const int run = (int)(blockIdx.x - n * p.runs);
    const int slot = threadIdx.x / cu, cl = (threadIdx.x - slot * cu) * V, c = run * p.cw + cl;
    const bool on = slot < slots;
    const int64_t rows = on ? p.L : 0;
    const int groups = p.cw / p.cg;
    float* gs = lds + slots * p.cw;
    const T* xp = static_cast<const T*>(p.x) + n * p.L * p.C + c;
    Unit<T, V> x[U];
    float sum[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = slot + (int64_t)i * slots;
        if (r < rows)
            x[i] = *reinterpret_cast<const Unit<T, V>*>(xp + r * p.C);
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (slot + (int64_t)i * slots < rows)
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += to_f32(x[i].e[j]);
    if (on)
#pragma unroll
        for (int j = 0; j < V; ++j) lds[slot * p.cw + cl + j] = sum[j];
    __syncthreads();
    group_sums(lds, slots, p.cw, p.cg, gs);
    __syncthreads();
    const float total = (float)p.L * (float)p.cg;
    float mean[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        mean[j] = gs[on ? (cl + j) / p.cg : 0] / total;  // (a division: a constant group's mean is exact)
        sum[j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (slot + (int64_t)i * slots < rows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = to_f32(x[i].e[j]) - mean[j];
                sum[j] = __builtin_fmaf(d, d, sum[j]);
            }
    if (on)
#pragma unroll
        for (int j = 0; j < V; ++j) lds[slot * p.cw + cl + j] = sum[j];
    __syncthreads();
    group_sums(lds, slots, p.cw, p.cg, gs + groups);
    __syncthreads();
    if ((int)threadIdx.x < groups) {
        const int64_t at = n * p.G + run * groups + threadIdx.x;
        p.mean[at] = gs[threadIdx.x] / total;
        p.rstd[at] = 1.0f / __builtin_sqrtf(gs[groups + threadIdx.x] / total + p.eps);
    }
    if (!on) return;
    float a[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        a[j] = 1.0f / __builtin_sqrtf(gs[groups + (cl + j) / p.cg] / total + p.eps);
        if (p.w) a[j] *= p.w[c + j];
        b[j] = p.b ? p.b[c + j] : 0.0f;
    }
    T* yp = static_cast<T*>(p.y) + n * p.L * p.C + c;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = slot + (int64_t)i * slots;
        if (r < rows) {
            Unit<T, V> y;
#pragma unroll
            for (int j = 0; j < V; ++j)
                y.e[j] = from_f32<T>(act_fwd(__builtin_fmaf(to_f32(x[i].e[j]) - mean[j], a[j], b[j]), p.act));
            *reinterpret_cast<Unit<T, V>*>(yp + r * p.C) = y;
        }
    }
}

template <typename T, int V, int U>
__global__ __launch_bounds__(512) void norm_slab_bwd_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const int cu = p.cw / V, slots = blockDim.x / cu;
    const int64_t n = blockIdx.x / p.runs;
    const int run = (int)(blockIdx.x - n * p.runs);
    const int slot = threadIdx.x / cu, cl = (threadIdx.x - slot * cu) * V, c = run * p.cw + cl;
    const bool on = slot < slots;
    const int64_t rows = on ? p.L : 0;
    const int groups = p.cw / p.cg;
    float *l1 = lds, *l2 = lds + slots * p.cw, *gs = l2 + slots * p.cw;
    const T* xp = static_cast<const T*>(p.x) + n * p.L * p.C + c;
    const T* dp = static_cast<const T*>(p.dy) + n * p.L * p.C + c;
    Unit<T, V> x[U], dy[U];
    float mean[V], rstd[V], w[V], b[V], s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = slot + (int64_t)i * slots;
        if (r < rows) {
            x[i] = *reinterpret_cast<const Unit<T, V>*>(xp + r * p.C);
            dy[i] = *reinterpret_cast<const Unit<T, V>*>(dp + r * p.C);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int64_t at = n * p.G + run * groups + (on ? (cl + j) / p.cg : 0);
        mean[j] = p.mean[at];
        rstd[j] = p.rstd[at];
        w[j] = p.w && on ? p.w[c + j] : 1.0f;
        b[j] = p.b && on ? p.b[c + j] : 0.0f;
        s1[j] = s2[j] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (slot + (int64_t)i * slots < rows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
                const float dz = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                s1[j] += dz;
                s2[j] = __builtin_fmaf(dz, xh, s2[j]);
            }
    if (on)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            l1[slot * p.cw + cl + j] = s1[j];
            l2[slot * p.cw + cl + j] = s2[j];
        }
    __syncthreads();
    // the channels' sums: to the workspace for the weights' gradients, and weighted for the group's
    for (int i = threadIdx.x; i < 2 * p.cw; i += blockDim.x) {
        float* l = i < p.cw ? l1 : l2;
        const int ch = i < p.cw ? i : i - p.cw;
        float v = 0.0f;
        for (int k = 0; k < slots; ++k) v += l[k * p.cw + ch];
        const int cc = run * p.cw + ch;
        if (p.part) p.part[(n * 2 + (i < p.cw ? 0 : 1)) * p.C + cc] = v;
        l[ch] = p.w ? v * p.w[cc] : v;
    }
    __syncthreads();
    group_sums(l1, 1, p.cw, p.cg, gs);
    group_sums(l2, 1, p.cw, p.cg, gs + groups);
    __syncthreads();
    if (!on) return;
    const float inv = 1.0f / ((float)p.L * (float)p.cg);
    float m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        m1[j] = gs[(cl + j) / p.cg] * inv;
        m2[j] = gs[groups + (cl + j) / p.cg] * inv;
    }
    T* yp = static_cast<T*>(p.y) + n * p.L * p.C + c;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int64_t r = slot + (int64_t)i * slots;
        if (r < rows) {
            Unit<T, V> y;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
                const float dz = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                y.e[j] = from_f32<T>(rstd[j] * (dz * w[j] - m1[j] - xh * m2[j]));
            }
            *reinterpret_cast<Unit<T, V>*>(yp + r * p.C) = y;
        }
    }
}

// ------------------------------------------------------------------------------------------------ two passes
constexpr int kBatch = 8;  // rows a thread has in flight

// First pass: per-channel sums of one row range.  Forward: the mean and the squares about it; backward: sum dz
// and sum dz xh.  LDS: [slots][2][units of the tile].
template <typename T, int V, bool BWD>
__global__ __launch_bounds__(256) void norm_sums_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const int64_t unit = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - unit * p.tiles);
    const int64_t n = unit / p.splits;
    const int split = (int)(unit - n * p.splits);
    const int cu = min(p.tunits, p.C / V - tile * p.tunits);
    const int slots = blockDim.x / cu, cw = cu * V;
    const int slot = threadIdx.x / cu, cl = (threadIdx.x - slot * cu) * V, c = tile * p.tunits * V + cl;
    const bool on = slot < slots;
    const int64_t r0 = split * p.srows, r1 = min(p.L, r0 + p.srows);
    float s1[V], s2[V], mean[V], rstd[V], w[V], b[V];
    float count = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        s1[j] = s2[j] = 0.0f;
        if (BWD) {
            const int64_t at = n * p.G + (on ? (c + j) / p.cg : 0);
            mean[j] = p.mean[at];
            rstd[j] = p.rstd[at];
            w[j] = p.w && on ? p.w[c + j] : 1.0f;
            b[j] = p.b && on ? p.b[c + j] : 0.0f;
        }
    }
    if (on) {
        const T* xp = static_cast<const T*>(p.x) + n * p.L * p.C + c;
        const T* dp = BWD ? static_cast<const T*>(p.dy) + n * p.L * p.C + c : nullptr;
        int64_t r = r0 + slot;
        for (; r + (int64_t)(kBatch - 1) * slots < r1; r += (int64_t)kBatch * slots) {
            Unit<T, V> x[kBatch], dy[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                x[i] = *reinterpret_cast<const Unit<T, V>*>(xp + (r + (int64_t)i * slots) * p.C);
                if (BWD) dy[i] = *reinterpret_cast<const Unit<T, V>*>(dp + (r + (int64_t)i * slots) * p.C);
            }
            const float join = count * kBatch / (count + kBatch), step = kBatch / (count + kBatch);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (BWD) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
                        const float dz = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                        s1[j] += dz;
                        s2[j] = __builtin_fmaf(dz, xh, s2[j]);
                    }
                } else {
                    float m = 0.0f, q = 0.0f;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) m += to_f32(x[i].e[j]);
                    m *= 1.0f / kBatch;
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float d = to_f32(x[i].e[j]) - m;
                        q = __builtin_fmaf(d, d, q);
                    }
                    // union of `count` values (s1 their mean, s2 their squares) and the batch
                    const float d = m - s1[j];
                    s1[j] = __builtin_fmaf(d, step, s1[j]);
                    s2[j] += __builtin_fmaf(d * d, join, q);
                }
            }
            count += kBatch;
        }
        for (; r < r1; r += slots) {
            const Unit<T, V> x = *reinterpret_cast<const Unit<T, V>*>(xp + r * p.C);
            Unit<T, V> dy;
            if (BWD) dy = *reinterpret_cast<const Unit<T, V>*>(dp + r * p.C);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (BWD) {
                    const float xh = (to_f32(x.e[j]) - mean[j]) * rstd[j];
                    const float dz = act_bwd(to_f32(dy.e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                    s1[j] += dz;
                    s2[j] = __builtin_fmaf(dz, xh, s2[j]);
                } else {
                    const float d = to_f32(x.e[j]) - s1[j];
                    s1[j] += d / (count + 1.0f);
                    s2[j] = __builtin_fmaf(d * d, count / (count + 1.0f), s2[j]);
                }
            }
            count += 1.0f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            lds[(slot * 2) * cw + cl + j] = s1[j];
            lds[(slot * 2 + 1) * cw + cl + j] = s2[j];
        }
        if (cl == 0) lds[slots * 2 * cw + slot] = count;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cw; i += blockDim.x) {
        float a = lds[i], q = lds[cw + i], k = lds[slots * 2 * cw];
        for (int s = 1; s < slots; ++s) {
            const float m = lds[s * 2 * cw + i], t = lds[(s * 2 + 1) * cw + i], ks = lds[slots * 2 * cw + s];
            if (BWD) {
                a += m;
                q += t;
            } else if (ks > 0.0f) {
                const float d = m - a;
                a = __builtin_fmaf(d, ks / (k + ks), a);
                q += t + d * d * (k * ks / (k + ks));
                k += ks;
            }
        }
        float* out = p.part + ((n * p.splits + split) * 2) * p.C + tile * p.tunits * V + i;
        out[0] = a;
        out[p.C] = q;
    }
}

// Joins the ranges and the channels of a group (a wave to a group).  Forward: mean and rstd; backward: m1, m2.
template <bool BWD>
__global__ __launch_bounds__(256) void norm_join_kernel(const NormParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t id = blockIdx.x * (int64_t)(blockDim.x >> 6) + (threadIdx.x >> 6);
    if (id >= p.N * p.G) return;
    const int64_t n = id / p.G;
    const int g = (int)(id - n * p.G);
    const float* part = p.part + n * p.splits * 2 * p.C + g * p.cg;
    const int entries = p.splits * p.cg;
    const float total = (float)p.L * (float)p.cg;
    float s = 0.0f, t = 0.0f;
    for (int i = lane; i < entries; i += 64) {
        const int split = i / p.cg, c = i - split * p.cg;
        const int64_t rows = min(p.L - split * p.srows, p.srows);
        const float m = part[(int64_t)split * 2 * p.C + c];
        if (BWD) {
            const float w = p.w ? p.w[g * p.cg + c] : 1.0f;
            s = __builtin_fmaf(w, m, s);
            t = __builtin_fmaf(w, part[((int64_t)split * 2 + 1) * p.C + c], t);
        } else {
            s = __builtin_fmaf((float)rows, m, s);
        }
    }
    s = wave_sum(s) / total;
    if (BWD) {
        t = wave_sum(t) / total;
        if (lane == 0) {
            p.gsum[id * 2] = s;
            p.gsum[id * 2 + 1] = t;
        }
        return;
    }
    for (int i = lane; i < entries; i += 64) {
        const int split = i / p.cg, c = i - split * p.cg;
        const int64_t rows = min(p.L - split * p.srows, p.srows);
        const float d = part[(int64_t)split * 2 * p.C + c] - s;
        t += __builtin_fmaf(d * d, (float)rows, part[((int64_t)split * 2 + 1) * p.C + c]);
    }
    t = wave_sum(t) / total;
    if (lane == 0) {
        p.mean[id] = s;
        p.rstd[id] = 1.0f / __builtin_sqrtf(t + p.eps);
    }
}

// Second pass: every value from its group's statistics.
template <typename T, int V, bool BWD>
__global__ __launch_bounds__(256) void norm_apply_kernel(const NormParams p) {
    const int64_t unit = blockIdx.x / p.tiles;
    const int tile = (int)(blockIdx.x - unit * p.tiles);
    const int64_t n = unit / p.splits;
    const int split = (int)(unit - n * p.splits);
    const int cu = min(p.tunits, p.C / V - tile * p.tunits);
    const int slots = blockDim.x / cu;
    const int slot = threadIdx.x / cu, c = (tile * p.tunits + (int)threadIdx.x - slot * cu) * V;
    if (slot >= slots) return;
    const int64_t r0 = split * p.srows, r1 = min(p.L, r0 + p.srows);
    float mean[V], rstd[V], w[V], b[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int64_t at = n * p.G + (c + j) / p.cg;
        mean[j] = p.mean[at];
        rstd[j] = p.rstd[at];
        w[j] = p.w ? p.w[c + j] : 1.0f;
        b[j] = p.b ? p.b[c + j] : 0.0f;
        if (BWD) {
            m1[j] = p.gsum[at * 2];
            m2[j] = p.gsum[at * 2 + 1];
        }
    }
    const int64_t base = n * p.L * p.C + c;
    const T *xp = static_cast<const T*>(p.x) + base, *dp = BWD ? static_cast<const T*>(p.dy) + base : nullptr;
    T* yp = static_cast<T*>(p.y) + base;
    constexpr int B = 4;
    for (int64_t r = r0 + slot; r < r1; r += (int64_t)B * slots) {
        Unit<T, V> x[B], dy[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (r + (int64_t)i * slots < r1) {
                x[i] = *reinterpret_cast<const Unit<T, V>*>(xp + (r + (int64_t)i * slots) * p.C);
                if (BWD) dy[i] = *reinterpret_cast<const Unit<T, V>*>(dp + (r + (int64_t)i * slots) * p.C);
            }
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (r + (int64_t)i * slots < r1) {
                Unit<T, V> y;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
                    const float z = __builtin_fmaf(xh, w[j], b[j]);
                    if (BWD) {
                        const float dz = act_bwd(to_f32(dy[i].e[j]), z, p.act);
                        y.e[j] = from_f32<T>(rstd[j] * (dz * w[j] - m1[j] - xh * m2[j]));
                    } else {
                        y.e[j] = from_f32<T>(act_fwd(z, p.act));
                    }
                }
                *reinterpret_cast<Unit<T, V>*>(yp + (r + (int64_t)i * slots) * p.C) = y;
            }
    }
}

// dw, db: the channels' sums over samples and ranges.  A workgroup to 64 channels, 16 threads down each.
__global__ __launch_bounds__(1024) void norm_weights_kernel(const NormParams p, int64_t parts) {
    __shared__ float red[2][16][64];
    const int cl = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + cl;
    float a = 0.0f, b = 0.0f;
    if (c < p.C)
        for (int64_t i = k; i < parts; i += 16) {
            b += p.part[i * 2 * p.C + c];
            a += p.part[(i * 2 + 1) * p.C + c];
        }
    red[0][k][cl] = a;
    red[1][k][cl] = b;
    __syncthreads();
    if (k < 2 && c < p.C) {
        float v = 0.0f;
        for (int i = 0; i < 16; ++i) v += red[k][i][cl];
        float* out = k == 0 ? p.dw : p.db;
        if (out) out[c] = v;
    }
}

template <typename T, int V, int U>
hipError_t launch_slab(const NormParams& p, bool bwd, hipStream_t s) {
    const int slots = p.threads / (p.cw / V);
    const size_t lds = ((size_t)slots * p.cw * (bwd ? 2 : 1) + 2 * (p.cw / p.cg)) * 4;
    const dim3 grid((unsigned)(p.N * p.runs));
    if (bwd)
        hipLaunchKernelGGL((norm_slab_bwd_kernel<T, V, U>), grid, dim3(p.threads), lds, s, p);
    else
        hipLaunchKernelGGL((norm_slab_fwd_kernel<T, V, U>), grid, dim3(p.threads), lds, s, p);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_v(const NormParams& p, bool bwd, hipStream_t s) {
    hipError_t e;
    if (p.slab) {
        e = p.units <= 1 ? launch_slab<T, V, 1>(p, bwd, s)
            : p.units <= 2 ? launch_slab<T, V, 2>(p, bwd, s)
            : p.units <= 4 ? launch_slab<T, V, 4>(p, bwd, s)
                           : launch_slab<T, V, 8>(p, bwd, s);
    } else {
        const dim3 grid((unsigned)(p.N * p.splits * p.tiles));
        // the last tile may be narrower and so have more slots; slots x channels never exceeds threads x V
        const size_t lds = ((size_t)2 * p.threads * V + p.threads) * 4;
        const dim3 jgrid((unsigned)((p.N * p.G + 3) / 4));
        if (bwd) {
            hipLaunchKernelGGL((norm_sums_kernel<T, V, true>), grid, dim3(p.threads), lds, s, p);
            hipLaunchKernelGGL((norm_join_kernel<true>), jgrid, dim3(256), 0, s, p);
            hipLaunchKernelGGL((norm_apply_kernel<T, V, true>), grid, dim3(p.threads), 0, s, p);
        } else {
            hipLaunchKernelGGL((norm_sums_kernel<T, V, false>), grid, dim3(p.threads), lds, s, p);
            hipLaunchKernelGGL((norm_join_kernel<false>), jgrid, dim3(256), 0, s, p);
            hipLaunchKernelGGL((norm_apply_kernel<T, V, false>), grid, dim3(p.threads), 0, s, p);
        }
        e = hipGetLastError();
    }
    if (e != hipSuccess || !bwd || !(p.dw || p.db)) return e;
    hipLaunchKernelGGL(norm_weights_kernel, dim3((unsigned)((p.C + 63) / 64)), dim3(1024), 0, s, p,
                       p.N * (p.slab ? 1 : (int64_t)p.splits));
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const NormParams& p, bool bwd, hipStream_t s) {
    return p.vec > 1 ? launch_v<T, 16 / sizeof(T)>(p, bwd, s) : launch_v<T, 1>(p, bwd, s);
}

}  // namespace

int64_t plan_norm(NormParams& p, int io_bytes, bool aligned, bool backward) {
    p.cg = p.C / p.G;
    const int v = 16 / io_bytes;
    p.vec = aligned && p.C % v == 0 ? v : 1;
    // Slab: the narrowest run of whole groups that is whole units, widened to full 128-byte lines while a thread
    // still holds at most eight units; the smallest workgroup that does.
    p.slab = 0;
    // (two tensors backward: half the threads, twice the registers)
    constexpr int kUnits = 8;
    const int kThreads = backward ? 512 : 1024;
    for (int k = 1; k <= p.G; ++k) {
        if (p.G % k || (k * p.cg) % p.vec) continue;
        const int64_t cu = (int64_t)k * p.cg / p.vec;
        if (cu > kThreads || p.L > (kThreads / cu) * (int64_t)kUnits) break;
        p.slab = 1;
        p.cw = k * p.cg;
        if ((int64_t)p.cw * io_bytes >= 128) break;
    }
    if (p.slab) {
        const int cu = p.cw / p.vec;
        p.runs = p.C / p.cw;
        for (p.threads = 64; p.threads < kThreads; p.threads *= 2)
            if (p.threads >= cu && p.L <= (p.threads / cu) * (int64_t)(p.threads < 256 ? 4 : kUnits)) break;
        const int slots = p.threads / cu;
        p.units = (int)((p.L + slots - 1) / slots);
        return backward && (p.dw || p.db) ? p.N * 2 * p.C * 4 : 0;
    }
    p.threads = 256;
    const int cu = p.C / p.vec;
    p.tiles = (cu + p.threads - 1) / p.threads;
    p.tunits = (cu + p.tiles - 1) / p.tiles;
    p.tiles = (cu + p.tunits - 1) / p.tunits;
    // about eight workgroups to a compute unit, ranges of at least 16 rows a slot
    const int64_t want = (2048 + p.N * p.tiles - 1) / (p.N * p.tiles);
    const int64_t slots = p.threads / p.tunits, floor_rows = slots * 16;
    int64_t splits = (p.L + floor_rows - 1) / floor_rows;
    if (splits > want) splits = want;
    if (splits < 1) splits = 1;
    p.srows = (p.L + splits - 1) / splits;
    p.splits = (int)((p.L + p.srows - 1) / p.srows);
    return p.N * p.splits * 2 * (int64_t)p.C * 4 + (backward ? p.N * p.G * 8 : 0);
}

hipError_t launch_group_norm_fwd(const NormParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_t<float>(p, false, s) : launch_t<__bf16>(p, false, s);
}

hipError_t launch_group_norm_bwd(const NormParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_t<float>(p, true, s) : launch_t<__bf16>(p, true, s);
}

}  // namespace sfm
