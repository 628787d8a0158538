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
//   store (one read, one write, one launch).  Threads take the means of their own values and the squares about them,
//   which are joined exactly, so a mean far from zero costs no digits.  256 x 198 x 320 bfloat16, 5 groups: 18 us,
//   3.6 TB/s; backward at 256 x 51 x 640, 10 groups: 18 us, 2.8 TB/s, and 4 for the weights (load, sums, store in
//   turn: what one workgroup waits for, the others of the unit hide in part).  Samples of a token fill few of a
//   workgroup's lanes (a run of 64 channels 8 of 64), and each leaves its channels' sums for the weights: 50688 tokens
//   of 320 channels, 5 groups, 231 us forward; backward 278, and 144 for the weights from 130 MB of sums.
// * Two passes, where a group does not fit: row ranges of a sample to separate workgroups, which leave per-channel
//   sums; a small kernel joins them in a fixed order; the second pass reads the input again (from the last-level
//   cache if it fits there).  Squares are taken about the mean of each batch of eight rows, and batches, channels
//   and ranges are joined by the exact formula for the squares of a union, again so that a large mean costs nothing.
//   16 x 12544 x 160 bfloat16, 32 groups: 48 us for 192 MB (16 sums, 5 join, 27 apply); backward at 4 x 12544 x 320
//   float32: 73 us for 321 MB (29, 5, 34, 5 the weights').
// Sums are float32 in a fixed order: repeated calls give the same bits.
#include <algorithm>

#include "delta_mma.h"
#include "sfm_norm.h"

namespace sfm {

namespace {

template <typename T, int V> struct alignas(V * sizeof(T)) Unit {
    T e[V];
};

// sigmoid without overflow: exp2 of a large positive argument is infinity and 1 / infinity is 0 (the reciprocal
// instruction, one unit in the last place: a full division costs ten times as much, more than all else here)
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-z * kLog2e)); }

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

// Groups of V neighbouring channels from `first` on (relative to where groups are counted from).
template <int V> struct GroupOf {
    int g[V];
    __device__ __forceinline__ GroupOf(int first, int cg) {
        int q = first / cg, r = first - q * cg;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            g[j] = q;
            if (++r == cg) r = 0, ++q;
        }
    }
};

// A wave's share of a group's entries in [slots][width] arrays, `eg` neighbours to a group: f(slot, column).
template <typename F> __device__ __forceinline__ void each_entry(int slots, int eg, int g, F f) {
    const int lane = threadIdx.x & 63;
    const int per = eg < 64 ? 64 / eg : 1;  // slots a wave takes at once
    const int ls = eg < 64 ? lane / eg : 0, lc = lane - ls * eg;
    if (ls >= per) return;
    for (int s = ls; s < slots; s += per)
        for (int c = lc; c < eg; c += 64) f(s, g * eg + c);
}

// Units of a sample's rows as a buffer: zeros past the last row, and stores there are dropped.
template <typename T, int V> __device__ __forceinline__ Unit<T, V> unit_load(const Buf& b, unsigned at) {
    if constexpr (V * sizeof(T) == 16) {
        typedef unsigned word __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(Unit<T, V>, buf_load<word>(b, at));
    } else {
        return __builtin_bit_cast(Unit<T, V>, buf_load<T>(b, at));
    }
}
template <typename T, int V> __device__ __forceinline__ void unit_store(const Buf& b, unsigned at, const Unit<T, V>& u) {
    if constexpr (V * sizeof(T) == 16) {
        typedef unsigned word __attribute__((ext_vector_type(4)));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(word, u), b.r, at, 0, 0);
    } else {
        buf_store<T>(b, at, u.e[0]);
    }
}

// ------------------------------------------------------------------------------------------------ slab kernels
// LDS, forward: [slots][entries] sums, means and squares about them (an entry is a thread's unit where units do not
// straddle groups, else a channel), row counts by slot, the groups' mean and 1 / deviation; backward: [slots][cw]
// sums of dz and of dz xh, then the groups'.
template <typename T, int V, int U, int THREADS, bool WHOLE>
__global__ __launch_bounds__(THREADS, 4) void norm_slab_fwd_kernel(const NormParams p) {
    constexpr int NE = WHOLE ? 1 : V;
    extern __shared__ float lds[];
    const int cu = p.cw / V, slots = blockDim.x / cu, ew = cu * NE, eg = p.cg / (V / NE);
    const int64_t n = blockIdx.x / p.runs;
    const int run = (int)(blockIdx.x - n * p.runs);
    const int slot = threadIdx.x / cu, u = threadIdx.x - slot * cu, cl = u * V, c = run * p.cw + cl;
    const bool on = slot < slots;
    const int groups = p.cw / p.cg;
    float *ls = lds, *lm = ls + slots * ew, *lq = lm + slots * ew, *lr = lq + slots * ew, *gm = lr + slots, *gr = gm + groups;
    const Buf xb = make_buf(static_cast<const T*>(p.x) + n * p.L * p.C, p.L * p.C * (int)sizeof(T));
    const unsigned at = on ? (unsigned)(slot * p.C + c) * (unsigned)sizeof(T) : kNowhere, step = (unsigned)(slots * p.C) * (unsigned)sizeof(T);
    Unit<T, V> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = unit_load<T, V>(xb, at + i * step);
    float w[V], b[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        w[j] = p.w && on ? p.w[c + j] : 1.0f;
        b[j] = p.b && on ? p.b[c + j] : 0.0f;
    }
    // this thread's rows, then the sums over them, their mean and the squares about it
    const int rows = on && slot < p.L ? ((int)p.L - 1 - slot) / slots + 1 : 0;
    float s[NE], m[NE], q[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) s[j] = q[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) s[j % NE] += to_f32(x[i].e[j]);
    const float count = (float)(rows * (V / NE));
#pragma unroll
    for (int j = 0; j < NE; ++j) m[j] = rows > 0 ? s[j] / count : 0.0f;
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (i < rows)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = to_f32(x[i].e[j]) - m[j % NE];
                q[j % NE] = __builtin_fmaf(d, d, q[j % NE]);
            }
    if (on) {
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            const int e = slot * ew + u * NE + j;
            ls[e] = s[j];
            lm[e] = m[j];
            lq[e] = q[j];
        }
        if (u == 0) lr[slot] = count;
    }
    __syncthreads();
    const float total = (float)p.L * (float)p.cg;
    for (int g = threadIdx.x >> 6; g < groups; g += blockDim.x >> 6) {
        float v = 0.0f;
        each_entry(slots, eg, g, [&](int k, int e) { v += ls[k * ew + e]; });
        const float mean = wave_sum(v) / total;  // (a division: a constant group's mean is exact)
        v = 0.0f;
        each_entry(slots, eg, g, [&](int k, int e) {
            const float n = lr[k], d = lm[k * ew + e] - mean;
            v += __builtin_fmaf(d * n, d, lq[k * ew + e]);  // (in this order: a slot without rows adds 0 whatever the mean)
        });
        const float rstd = 1.0f / __builtin_sqrtf(wave_sum(v) / total + p.eps);
        if ((threadIdx.x & 63) == 0) {
            gm[g] = mean;
            gr[g] = rstd;
            p.mean[n * p.G + run * groups + g] = mean;
            p.rstd[n * p.G + run * groups + g] = rstd;
        }
    }
    __syncthreads();
    float mean[V];
    if constexpr (WHOLE) {
        const int g = on ? cl / p.cg : 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mean[j] = gm[g];
            w[j] *= gr[g];
        }
    } else {
        const GroupOf<V> grp(on ? cl : 0, p.cg);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            mean[j] = gm[grp.g[j]];
            w[j] *= gr[grp.g[j]];
        }
    }
    const Buf yb = make_buf(static_cast<T*>(p.y) + n * p.L * p.C, p.L * p.C * (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < U; ++i) {
        Unit<T, V> y;
#pragma unroll
        for (int j = 0; j < V; ++j)
            y.e[j] = from_f32<T>(act_fwd(__builtin_fmaf(to_f32(x[i].e[j]) - mean[j], w[j], b[j]), p.act));
        unit_store<T, V>(yb, at + i * step, y);
    }
}

template <typename T, int V, int U, int THREADS>
__global__ __launch_bounds__(THREADS, (U <= 4 ? 3 : 2)) void norm_slab_bwd_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const int cu = p.cw / V, slots = blockDim.x / cu;
    const int64_t n = blockIdx.x / p.runs;
    const int run = (int)(blockIdx.x - n * p.runs);
    const int slot = threadIdx.x / cu, cl = (threadIdx.x - slot * cu) * V, c = run * p.cw + cl;
    const bool on = slot < slots;
    const int groups = p.cw / p.cg;
    float *l1 = lds, *l2 = lds + slots * p.cw, *gs = l2 + slots * p.cw, *gq = gs + groups;
    const GroupOf<V> grp(on ? cl : 0, p.cg);
    const Buf xb = make_buf(static_cast<const T*>(p.x) + n * p.L * p.C, p.L * p.C * (int)sizeof(T));
    const Buf db = make_buf(static_cast<const T*>(p.dy) + n * p.L * p.C, p.L * p.C * (int)sizeof(T));
    const unsigned at = on ? (unsigned)(slot * p.C + c) * (unsigned)sizeof(T) : kNowhere, step = (unsigned)(slots * p.C) * (unsigned)sizeof(T);
    Unit<T, V> x[U], dy[U];
    float mean[V], rstd[V], w[V], b[V], s1[V], s2[V], dz[U][V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        x[i] = unit_load<T, V>(xb, at + i * step);
        dy[i] = unit_load<T, V>(db, at + i * step);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int64_t ga = n * p.G + run * groups + grp.g[j];
        mean[j] = p.mean[ga];
        rstd[j] = p.rstd[ga];
        w[j] = p.w && on ? p.w[c + j] : 1.0f;
        b[j] = p.b && on ? p.b[c + j] : 0.0f;
        s1[j] = s2[j] = 0.0f;
    }
    // (rows past the end are zeros: dz = 0)
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
            dz[i][j] = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
            s1[j] += dz[i][j];
            s2[j] = __builtin_fmaf(dz[i][j], xh, s2[j]);
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
#pragma unroll 8
        for (int k = 0; k < slots; ++k) v += l[k * p.cw + ch];
        const int cc = run * p.cw + ch;
        if (p.part) p.part[(n * 2 + (i < p.cw ? 0 : 1)) * p.C + cc] = v;
        l[ch] = p.w ? v * p.w[cc] : v;
    }
    __syncthreads();
    const float total = (float)p.L * (float)p.cg;
    for (int g = threadIdx.x >> 6; g < groups; g += blockDim.x >> 6) {
        float v1 = 0.0f, v2 = 0.0f;
        each_entry(1, p.cg, g, [&](int, int e) {
            v1 += l1[e];
            v2 += l2[e];
        });
        v1 = wave_sum(v1);
        v2 = wave_sum(v2);
        if ((threadIdx.x & 63) == 0) {
            gs[g] = v1 / total;
            gq[g] = v2 / total;
        }
    }
    __syncthreads();
    const Buf yb = make_buf(static_cast<T*>(p.y) + n * p.L * p.C, p.L * p.C * (int)sizeof(T));
    // dx = rstd (w dz - m1 - xh m2) = (rstd w) dz - (rstd^2 m2) (x - mean) - rstd m1.  In a group of one value nothing
    // varies: its dx is zero, where the rounding of w dz - m1 by rstd, 1 / sqrt(eps) there, would be left.
    const float vary = p.L * p.cg > 1 ? 1.0f : 0.0f;
    float k2[V], k1[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        w[j] *= rstd[j] * vary;
        k2[j] = rstd[j] * rstd[j] * gq[grp.g[j]];
        k1[j] = rstd[j] * gs[grp.g[j]] * vary;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        Unit<T, V> y;
#pragma unroll
        for (int j = 0; j < V; ++j)
            y.e[j] = from_f32<T>(__builtin_fmaf(dz[i][j], w[j], -__builtin_fmaf(to_f32(x[i].e[j]) - mean[j], k2[j], k1[j])));
        unit_store<T, V>(yb, at + i * step, y);
    }
}

// ------------------------------------------------------------------------------------------------ two passes
constexpr int kBatch = 8;  // rows a thread has in flight

// Rows r0 .. r1 - 1 of sample n as a buffer that starts at row r0 (a range ends below 2^30 bytes: plan_norm).
template <typename T> __device__ __forceinline__ Buf range_buf(const void* x, const NormParams& p, int64_t n, int64_t r0, int64_t r1) {
    return make_buf(static_cast<const T*>(x) + (n * p.L + r0) * p.C, (r1 - r0) * p.C * (int)sizeof(T));
}

// First pass: per-channel sums of one row range.  Forward: the mean and the squares about it; backward: sum dz
// and sum dz xh.  LDS: [slots][2][channels of the tile], then row counts by slot.
template <typename T, int V, bool BWD>
__global__ __launch_bounds__(256) void norm_sums_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const unsigned unit = blockIdx.x / (unsigned)p.tiles, tile = blockIdx.x - unit * p.tiles;
    const unsigned n = unit / (unsigned)p.splits, split = unit - n * p.splits;
    const int cu = min(p.tunits, p.C / V - (int)tile * p.tunits);
    const int slots = blockDim.x / cu, cw = cu * V;
    const int slot = threadIdx.x / cu, cl = (threadIdx.x - slot * cu) * V, c = tile * p.tunits * V + cl;
    const bool on = slot < slots;
    const int64_t r0 = split * p.srows, r1 = min(p.L, r0 + p.srows);
    const int len = (int)(r1 - r0);
    float s1[V], s2[V], mean[V], rstd[V], w[V], b[V];
    float count = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s1[j] = s2[j] = 0.0f;
    if (BWD) {
        const GroupOf<V> grp(on ? c : 0, p.cg);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int64_t at = (int64_t)n * p.G + grp.g[j];
            mean[j] = p.mean[at];
            rstd[j] = p.rstd[at];
            w[j] = p.w && on ? p.w[c + j] : 1.0f;
            b[j] = p.b && on ? p.b[c + j] : 0.0f;
        }
    }
    const Buf xb = range_buf<T>(p.x, p, n, r0, r1), db = BWD ? range_buf<T>(p.dy, p, n, r0, r1) : xb;
    const unsigned step = (unsigned)(slots * p.C) * (unsigned)sizeof(T);
    unsigned at = on ? (unsigned)(slot * p.C + c) * (unsigned)sizeof(T) : kNowhere;
    for (int r = slot; r < len && on; r += kBatch * slots, at += kBatch * step) {
        Unit<T, V> x[kBatch], dy[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            x[i] = unit_load<T, V>(xb, at + i * step);
            if (BWD) dy[i] = unit_load<T, V>(db, at + i * step);
        }
        if (BWD) {  // (rows past the range are zeros: dz = 0)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float xh = (to_f32(x[i].e[j]) - mean[j]) * rstd[j];
                    const float dz = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                    s1[j] += dz;
                    s2[j] = __builtin_fmaf(dz, xh, s2[j]);
                }
        } else {
            // the batch by itself, then the union of it and the `count` values before (s1 their mean, s2 their squares)
            const int rows = min(kBatch, (len - 1 - r) / slots + 1);
            const float nb = (float)rows, all = count + nb, join = count * nb / all, part = nb / all, inv = 1.0f / nb;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float m = 0.0f, q = 0.0f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) m += to_f32(x[i].e[j]);
                m *= inv;
                if (rows == kBatch) {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float d = to_f32(x[i].e[j]) - m;
                        q = __builtin_fmaf(d, d, q);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kBatch; ++i) {
                        const float d = i < rows ? to_f32(x[i].e[j]) - m : 0.0f;
                        q = __builtin_fmaf(d, d, q);
                    }
                }
                const float d = m - s1[j];
                s1[j] = __builtin_fmaf(d, part, s1[j]);
                s2[j] += __builtin_fmaf(d * join, d, q);  // (in this order: 0 for the first batch, also where d * d overflows)
            }
            count = all;
        }
    }
    if (on) {
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
        float* out = p.part + (((int64_t)n * p.splits + split) * 2) * p.C + tile * p.tunits * V + i;
        out[0] = a;
        out[p.C] = q;
    }
}

// Joins the ranges of a sample's channels: a workgroup to 16 channels, 16 threads down the ranges of each.  The
// result takes the place of the first range's sums.
template <bool BWD>
__global__ __launch_bounds__(256) void norm_join_kernel(const NormParams p, unsigned tiles) {
    __shared__ float l1[16][17], l2[16][17], lk[16];
    const unsigned n = blockIdx.x / tiles;
    const int cl = threadIdx.x & 15, k = threadIdx.x >> 4, c = (int)(blockIdx.x - n * tiles) * 16 + cl;
    float* part = p.part + (int64_t)n * p.splits * 2 * p.C + c;
    float a = 0.0f, q = 0.0f, count = 0.0f;
    if (c < p.C)
#pragma unroll 4
        for (int i = k; i < p.splits; i += 16) {
            const float m = part[(int64_t)i * 2 * p.C], t = part[((int64_t)i * 2 + 1) * p.C];
            if (BWD) {
                a += m;
                q += t;
            } else {
                const float rows = (float)min(p.L - i * p.srows, p.srows), d = m - a;
                a = __builtin_fmaf(d, rows / (count + rows), a);
                q += t + d * (count * rows / (count + rows)) * d;  // (0 for the first range)
                count += rows;
            }
        }
    l1[k][cl] = a;
    l2[k][cl] = q;
    if (cl == 0) lk[k] = count;
    __syncthreads();
    if (k != 0 || c >= p.C) return;
    for (int i = 1; i < 16; ++i) {
        const float m = l1[i][cl], t = l2[i][cl], rows = lk[i];
        if (BWD) {
            a += m;
            q += t;
        } else if (rows > 0.0f) {
            const float d = m - a;
            a = __builtin_fmaf(d, rows / (count + rows), a);
            q += t + d * d * (count * rows / (count + rows));
            count += rows;
        }
    }
    part[0] = a;
    part[p.C] = q;
}

// Joins the channels of group g (channels `lane`, `lane` + `step`, .. of it, summed by `sum`): forward mean and
// 1 / deviation, backward m1 and m2.
template <bool BWD, typename Sum>
__device__ __forceinline__ void join_group(const NormParams& p, const float* part, int g, int lane, int step, Sum sum, float& r1, float& r2) {
    const float total = (float)p.L * (float)p.cg;
    float s = 0.0f, t = 0.0f;
#pragma unroll 4
    for (int c = lane; c < p.cg; c += step) {
        const float w = BWD && p.w ? p.w[g * p.cg + c] : 1.0f;
        s = __builtin_fmaf(w, part[g * p.cg + c], s);
        if (BWD) t = __builtin_fmaf(w, part[p.C + g * p.cg + c], t);
    }
    if (BWD) {
        r1 = sum(s) / total;
        r2 = sum(t) / total;
        return;
    }
    r1 = sum(s) / (float)p.cg;
#pragma unroll 4
    for (int c = lane; c < p.cg; c += step) {
        const float d = part[g * p.cg + c] - r1;
        t += __builtin_fmaf(d * d, (float)p.L, part[p.C + g * p.cg + c]);
    }
    r2 = 1.0f / __builtin_sqrtf(sum(t) / total + p.eps);
}

// Second pass: the tile's groups from their channels' sums (every workgroup for itself: a few loads), then every
// value from its group's.  LDS: two floats to a group of the tile.
template <typename T, int V, bool BWD>
__global__ __launch_bounds__(256) void norm_apply_kernel(const NormParams p) {
    extern __shared__ float lds[];
    const unsigned unit = blockIdx.x / (unsigned)p.tiles, tile = blockIdx.x - unit * p.tiles;
    const unsigned n = unit / (unsigned)p.splits, split = unit - n * p.splits;
    const int cu = min(p.tunits, p.C / V - (int)tile * p.tunits);
    const int slots = blockDim.x / cu;
    const int slot = threadIdx.x / cu, c0 = tile * p.tunits * V, c = c0 + ((int)threadIdx.x - slot * cu) * V;
    const bool on = slot < slots;
    const int64_t r0 = split * p.srows, r1 = min(p.L, r0 + p.srows);
    const int len = (int)(r1 - r0);
    const Buf xb = range_buf<T>(p.x, p, n, r0, r1), db = BWD ? range_buf<T>(p.dy, p, n, r0, r1) : xb, yb = range_buf<T>(p.y, p, n, r0, r1);
    const unsigned step = (unsigned)(slots * p.C) * (unsigned)sizeof(T);
    unsigned at = on ? (unsigned)(slot * p.C + c) * (unsigned)sizeof(T) : kNowhere;
    constexpr int B = 4;
    Unit<T, V> x[B], dy[B];
    auto fetch = [&] {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            x[i] = unit_load<T, V>(xb, at + i * step);
            if (BWD) dy[i] = unit_load<T, V>(db, at + i * step);
        }
    };
    fetch();  // on their way while the groups are joined
    const int g0 = c0 / p.cg, groups = (c0 + cu * V - 1) / p.cg - g0 + 1;
    {
        const float* part = p.part + (int64_t)n * p.splits * 2 * p.C;
        auto put = [&](int g, float a, float b) {
            lds[g] = a;
            lds[groups + g] = b;
            if (!BWD && split == 0 && (g0 + g) * p.cg >= c0) {
                p.mean[(int64_t)n * p.G + g0 + g] = a;
                p.rstd[(int64_t)n * p.G + g0 + g] = b;
            }
        };
        float a, b;
        if (p.cg <= 32) {
            for (int g = threadIdx.x; g < groups; g += blockDim.x) {
                join_group<BWD>(p, part, g0 + g, 0, 1, [](float v) { return v; }, a, b);
                put(g, a, b);
            }
        } else {
            for (int g = threadIdx.x >> 6; g < groups; g += blockDim.x >> 6) {
                join_group<BWD>(p, part, g0 + g, threadIdx.x & 63, 64, wave_sum, a, b);
                if ((threadIdx.x & 63) == 0) put(g, a, b);
            }
        }
    }
    __syncthreads();
    if (!on) return;
    const GroupOf<V> grp(c, p.cg);
    float mean[V], rstd[V], w[V], b[V], m1[V], m2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int g = grp.g[j] - g0;
        w[j] = p.w ? p.w[c + j] : 1.0f;
        b[j] = p.b ? p.b[c + j] : 0.0f;
        if (BWD) {
            mean[j] = p.mean[(int64_t)n * p.G + grp.g[j]];
            rstd[j] = p.rstd[(int64_t)n * p.G + grp.g[j]];
            m1[j] = lds[g];
            m2[j] = lds[groups + g];
        } else {
            mean[j] = lds[g];
            w[j] *= lds[groups + g];
        }
    }
    for (int r = slot; r < len; r += B * slots) {
        Unit<T, V> y[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xd = to_f32(x[i].e[j]) - mean[j];
                if (BWD) {
                    const float xh = xd * rstd[j];
                    const float dz = act_bwd(to_f32(dy[i].e[j]), __builtin_fmaf(xh, w[j], b[j]), p.act);
                    y[i].e[j] = from_f32<T>(rstd[j] * (dz * w[j] - m1[j] - xh * m2[j]));
                } else {
                    y[i].e[j] = from_f32<T>(act_fwd(__builtin_fmaf(xd, w[j], b[j]), p.act));
                }
            }
        const unsigned here = at;
        at += B * step;
        fetch();
#pragma unroll
        for (int i = 0; i < B; ++i) unit_store<T, V>(yb, here + i * step, y[i]);
    }
}

// dw, db: the channels' sums over samples (`stride` floats apart).  A workgroup to 16 channels, 64 threads down each.
__global__ __launch_bounds__(1024) void norm_weights_kernel(const NormParams p, int64_t stride) {
    __shared__ float red[2][64][17];
    const int cl = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int c = blockIdx.x * 16 + cl;
    float a = 0.0f, b = 0.0f;
    if (c < p.C)
#pragma unroll 4
        for (int64_t i = k; i < p.N; i += 64) {
            b += p.part[i * stride + c];
            a += p.part[i * stride + p.C + c];
        }
    red[0][k][cl] = a;
    red[1][k][cl] = b;
    __syncthreads();
    for (int m = 32; m > 0; m >>= 1) {
        if (k < m) {
            red[0][k][cl] += red[0][k + m][cl];
            red[1][k][cl] += red[1][k + m][cl];
        }
        __syncthreads();
    }
    if (k < 2 && c < p.C) {
        float* out = k == 0 ? p.dw : p.db;
        if (out) out[c] = red[k][0][cl];
    }
}

template <typename T, int V, int U, int THREADS>
hipError_t launch_slab(const NormParams& p, bool bwd, hipStream_t s) {
    const int cu = p.cw / V, slots = p.threads / cu, groups = p.cw / p.cg;
    const dim3 grid((unsigned)(p.N * p.runs));
    if constexpr (THREADS <= 512)
        if (bwd) {
            const size_t lds = ((size_t)slots * p.cw * 2 + 2 * groups) * 4;
            hipLaunchKernelGGL((norm_slab_bwd_kernel<T, V, U, THREADS>), grid, dim3(p.threads), lds, s, p);
            return hipGetLastError();
        }
    const bool whole = p.cg % V == 0;
    const size_t lds = ((size_t)slots * (whole ? cu : p.cw) * 3 + slots + 2 * groups) * 4;
    auto kern = whole ? norm_slab_fwd_kernel<T, V, U, THREADS, true> : norm_slab_fwd_kernel<T, V, U, THREADS, false>;
    if (lds > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kern, grid, dim3(p.threads), lds, s, p);
    return hipGetLastError();
}

// The launches of one part of a call's samples.
template <typename T, int V>
hipError_t launch_samples(const NormParams& p, bool bwd, hipStream_t s) {
    if (p.slab)
        return p.threads > 512   ? launch_slab<T, V, 8, 1024>(p, bwd, s)
               : p.threads > 256 ? launch_slab<T, V, 8, 512>(p, bwd, s)
               : p.units <= 1    ? launch_slab<T, V, 1, 256>(p, bwd, s)
               : p.units <= 2    ? launch_slab<T, V, 2, 256>(p, bwd, s)
               : p.units <= 4    ? launch_slab<T, V, 4, 256>(p, bwd, s)
                                 : launch_slab<T, V, 8, 256>(p, bwd, s);
    const dim3 grid((unsigned)(p.N * p.splits * p.tiles));
    // the last tile may be narrower and so have more slots; slots x channels never exceeds threads x V
    const size_t lds = ((size_t)2 * p.threads * V + p.threads) * 4;
    const unsigned jt = (unsigned)((p.C + 15) / 16);
    const size_t glds = ((size_t)2 * (p.tunits * V / p.cg + 2)) * 4;
    hipLaunchKernelGGL((bwd ? norm_sums_kernel<T, V, true> : norm_sums_kernel<T, V, false>), grid, dim3(p.threads), lds, s, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.splits > 1) {  // (one range's sums are the sample's)
        hipLaunchKernelGGL((bwd ? norm_join_kernel<true> : norm_join_kernel<false>), dim3((unsigned)p.N * jt), dim3(256), 0, s, p, jt);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((bwd ? norm_apply_kernel<T, V, true> : norm_apply_kernel<T, V, false>), grid, dim3(p.threads), glds, s, p);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_v(const NormParams& p, bool bwd, hipStream_t s) {
    // A launch holds fewer than 2^32 work items: so many samples to one (2^20 tokens of 4096 channels in 64 groups, each
    // normed by itself, are 2^26 workgroups of 64).
    const int64_t wide = p.slab ? p.runs : std::max((int64_t)p.splits * p.tiles, (int64_t)(p.C + 15) / 16);
    const int64_t most = ((1LL << 32) - 1) / (p.slab ? p.threads : 256) / wide;
    const int64_t sums = 2 * (int64_t)p.C * (p.slab ? 1 : p.splits);  // floats a sample leaves in the workspace
    hipError_t e = hipSuccess;
    for (int64_t n = 0; n < p.N && e == hipSuccess; n += most) {
        NormParams q = p;
        const int64_t at = n * p.L * p.C * (int64_t)sizeof(T);
        q.x = static_cast<const char*>(p.x) + at;
        if (p.dy) q.dy = static_cast<const char*>(p.dy) + at;
        q.y = static_cast<char*>(p.y) + at;
        q.mean += n * p.G;
        q.rstd += n * p.G;
        if (p.part) q.part += n * sums;
        q.N = std::min(p.N - n, most);
        e = launch_samples<T, V>(q, bwd, s);
    }
    if (e != hipSuccess || !bwd || !(p.dw || p.db)) return e;
    hipLaunchKernelGGL(norm_weights_kernel, dim3((unsigned)((p.C + 15) / 16)), dim3(1024), 0, s, p, sums);
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
    // still holds at most eight units; the smallest workgroup that does (198 rows of 64 bfloat16 channels: 30 us a
    // 1280 runs with 256 threads of eight units, 39 us with 512 of four; what a thread does once costs more).
    p.slab = 0;
    // (two tensors backward: half the threads, twice the registers)
    constexpr int kUnits = 8;
    const int kThreads = backward ? 512 : 1024;
    for (int k = 1; k <= p.G; ++k) {
        if (p.G % k || (k * p.cg) % p.vec) continue;
        const int64_t cu = (int64_t)k * p.cg / p.vec;
        if (cu > kThreads || p.L > (kThreads / cu) * (int64_t)kUnits || p.L * p.C >= 1 << 28) break;
        p.slab = 1;
        p.cw = k * p.cg;
        if ((int64_t)p.cw * io_bytes >= 128) break;
    }
    if (p.slab) {
        const int cu = p.cw / p.vec;
        p.runs = p.C / p.cw;
        // (a wave joins its groups one after the other: four of them at most; 32 groups of 3 channels, 3 rows: 14 us a call, 32 with one wave)
        const int joiners = std::min(kThreads, (p.cw / p.cg + 3) / 4 * 64);
        for (p.threads = 64; p.threads < kThreads; p.threads *= 2)
            if (p.threads >= cu && p.threads >= joiners && p.L <= p.threads / cu * (int64_t)(p.threads < 256 ? 4 : kUnits)) break;
        const int slots = p.threads / cu;
        p.units = (int)((p.L + slots - 1) / slots);
        return backward && (p.dw || p.db) ? p.N * 2 * p.C * 4 : 0;
    }
    p.threads = 256;
    const int cu = p.C / p.vec;
    p.tiles = (cu + p.threads - 1) / p.threads;
    p.tunits = (cu + p.tiles - 1) / p.tiles;
    p.tiles = (cu + p.tunits - 1) / p.tunits;
    // about eight workgroups to a compute unit, ranges of at least 16 rows a slot and below 2^30 bytes
    const int64_t want = (2048 + p.N * p.tiles - 1) / (p.N * p.tiles);
    const int64_t slots = p.threads / p.tunits, floor_rows = slots * 16;
    int64_t splits = (p.L + floor_rows - 1) / floor_rows;
    if (splits > want) splits = want;
    const int64_t most = (1 << 28) / p.C, fewest = (p.L + most - 1) / most;
    if (splits < fewest) splits = fewest;
    p.srows = (p.L + splits - 1) / splits;
    p.splits = (int)((p.L + p.srows - 1) / p.srows);
    return p.N * p.splits * 2 * (int64_t)p.C * 4;
}

hipError_t launch_group_norm_fwd(const NormParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_t<float>(p, false, s) : launch_t<__bf16>(p, false, s);
}

hipError_t launch_group_norm_bwd(const NormParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_t<float>(p, true, s) : launch_t<__bf16>(p, true, s);
}

}  // namespace sfm
