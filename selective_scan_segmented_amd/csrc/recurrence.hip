// recurrence.hip -- the gated linear recurrence (gfx950): forward, backward and one token of many requests.
//
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// and with G_t = dy_t + a_{t+1} G_{t+1}, s = sigmoid, m = sqrt(1 - a^2), P = G la (a h_{t-1} - a^2 / m s(i) x):
//
//     dx = G m s(i),  di = dx x (1 - s(i)),  dr = P (1 - s(r)),  dlam = s(lam) / softplus(lam) sum P,  dh0 = a_0 G_0.
//
// Bound by memory: 8 bytes a bfloat16 value forward, 16 backward, against some 30 and 65 lane operations.  So every
// value is read once and a row is spread over as many lanes as it takes to keep the card's loads in flight: a lane
// holds 8 tokens of 4 bytes of channels in registers and finds what they make of a state, h -> A h + H; a lane a
// channel joins the chunks of a block through LDS; then every lane walks its 8 tokens from its own state.  Rows longer
// than a block hand their states on through words in memory (rec_block.h), so that they too are read once.
// The backward walks the same way back with u_t = a_{t+1} G_{t+1}: a u + a dy; it makes the gates again for its second
// look at the tokens, from what it holds in registers as it lies in memory.
#include "rec_block.h"

namespace sfm {

namespace {

constexpr int kThreads = 512;  // most to a workgroup of the rows' kernels

// One row (or block of one) of a lane: its chunk's place.
struct Chunk {
    int n;         // tokens of the block from the chunk's first on (0 or less: none)
    int64_t tok;   // the chunk's first token
    int ch;        // the lane's first channel
    bool live;     // has channels
};

template <typename T, int C>
__device__ __forceinline__ void load_chunk(RecPack<T, C> (&v)[kRecChunk], const void* base, int64_t ld, const Chunk& c, uint32_t none) {
    const T* p = static_cast<const T*>(base) + c.tok * ld + c.ch;
    if (c.live && c.n >= kRecChunk) {
#pragma unroll
        for (int t = 0; t < kRecChunk; ++t, p += ld) v[t].load(p);
    } else {
#pragma unroll
        for (int t = 0; t < kRecChunk; ++t, p += ld) {
            v[t].v = none;
            if (c.live && t < c.n) v[t].load(p);
        }
    }
}

// Joins the chunks' (A, H) of [rows][chunks][channels] in LDS: a lane a row and channel.  In their place: the state
// before every chunk.  BACK: chunks from the last to the first.
template <typename T, int C, bool MULTI, bool BACK>
__device__ __forceinline__ void join_chunks(const RecParams& p, float2* agg, const RecPlace& at, int64_t base_row, int blocks_of_row) {
    const RecPlan& q = p.plan;
    const int width = q.nc * C;
    for (int m = threadIdx.x; m < q.nr * width; m += blockDim.x) {
        const int rr = MULTI ? 0 : m / width, w = m - rr * width, ch = at.tile * width + w;
        const int64_t s = base_row + rr;
        if (ch >= p.D || s >= p.rows) continue;
        float2* a = agg + rr * q.nt * width + w;
        const float* before = BACK ? p.dhT : p.h0;
        float* after = BACK ? p.dh0 : p.hT;
        float h = 0.0f;
        const bool starts = !MULTI || at.block == (BACK ? blocks_of_row - 1 : 0);
        const bool ends = !MULTI || at.block == (BACK ? 0 : blocks_of_row - 1);
        if (starts && before) h = before[s * p.D + ch];
        if constexpr (MULTI) {
            const bool tells = !ends || p.offsets;  // (packed rows: always, rec_look_back)
            if (!starts || tells) {
                const int64_t stride = (int64_t)q.tiles * width;
                uint64_t* word = p.w_words + at.entry * stride + ch;
                float A = 1.0f, H = 0.0f;
                for (int k = 0; k < q.nt; ++k) {
                    const float2 v = a[(BACK ? q.nt - 1 - k : k) * width];
                    H = __builtin_fmaf(v.x, H, v.y);
                    A *= v.x;
                }
                if (!starts) {
                    if (tells) rec_publish(word, rec_factor(A), H);
                    h = rec_look_back<BACK>(BACK ? word + stride : word - stride, BACK ? stride : -stride,
                                      BACK ? blocks_of_row - 1 - at.block : at.block);
                }
                if (tells) rec_publish(word, kRecWhole, __builtin_fmaf(A, h, H));
            }
        }
        for (int k = 0; k < q.nt; ++k) {
            float2* v = a + (BACK ? q.nt - 1 - k : k) * width;
            const float2 f = *v;
            v->x = h;
            h = __builtin_fmaf(f.x, h, f.y);
        }
        if (ends && after) after[s * p.D + ch] = h;
    }
}

// The lane's place: rows side by side, in them chunks, in them channels.  Rows of several blocks: false where the
// workgroup has no tokens (its word says so).
template <typename T, int C, bool MULTI, bool BACK>
__device__ __forceinline__ bool lane_place(const RecParams& p, uint32_t* shared, RecPlace& at, int64_t& base_row, int& blocks_of_row,
                                           Chunk& c, int& slot, bool& row_start) {
    const RecPlan& q = p.plan;
    const int per_row = q.nc * q.nt;
    const int rr = MULTI ? 0 : (int)threadIdx.x / per_row;
    const int rest = (int)threadIdx.x - rr * per_row, tc = rest / q.nc, cl = rest - tc * q.nc;
    int64_t first = 0;
    int len = 0, skip = 0;
    if constexpr (MULTI) {
        at = rec_place<BACK>(p, shared, first, len);
        if (at.row < 0) return false;
        const int block = q.nt * kRecChunk;
        blocks_of_row = len > 0 ? (len + block - 1) / block : 1;
        base_row = at.row;
        skip = at.block * block;
        if (at.block >= blocks_of_row) {  // an entry of no row
            for (int m = threadIdx.x; m < q.nc * C; m += blockDim.x) {
                const int ch = at.tile * q.nc * C + m;
                rec_publish(p.w_words + at.entry * ((int64_t)q.tiles * q.nc * C) + ch, kRecWhole, 0.0f);
                if (BACK && ch < p.D) p.w_lam[at.entry * p.D + ch] = 0.0f;
            }
            return false;
        }
    } else {
        at.tile = blockIdx.x % (unsigned)q.tiles;
        at.entry = blockIdx.x / (unsigned)q.tiles;
        at.row = at.block = 0;
        base_row = at.entry * q.nr;
        blocks_of_row = 1;
        if (rr < q.nr && base_row + rr < p.rows) rec_row(p, (int)(base_row + rr), first, len);
    }
    const int t0 = skip + tc * kRecChunk;
    c.n = len - t0;
    if constexpr (MULTI) c.n = c.n < (q.nt - tc) * kRecChunk ? c.n : (q.nt - tc) * kRecChunk;
    c.tok = first + t0;
    c.ch = (at.tile * q.nc + cl) * C;
    c.live = rr < q.nr && c.ch < p.D;
    slot = (rr * q.nt + tc) * q.nc * C + cl * C;
    row_start = t0 == 0;
    return true;
}

template <typename T, int C, bool MULTI>
__global__ __launch_bounds__(kThreads, 4) void rec_fwd_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    __shared__ float2 agg[kThreads * C];
    __shared__ uint32_t shared[2];
    RecPlace at;
    int64_t base_row;
    int blocks_of_row, slot;
    Chunk c;
    bool row_start;
    if (!lane_place<T, C, MULTI, false>(p, shared, at, base_row, blocks_of_row, c, slot, row_start)) return;
    float a[kRecChunk][C], b[kRecChunk][C];
    {
        RecPack<T, C> r[kRecChunk], i[kRecChunk], x[kRecChunk];
        load_chunk<T, C>(r, p.r, p.ldr, c, RecPack<T, C>::kMinusInf);
        load_chunk<T, C>(i, p.i, p.ldi, c, 0);
        load_chunk<T, C>(x, p.x, p.ldx, c, 0);
        float rate[C], A[C], H[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            rate[j] = c.live ? rec_rate(p.lam[c.ch + j], p.c) : 0.0f;
            A[j] = 1.0f, H[j] = 0.0f;
        }
#pragma unroll
        for (int t = 0; t < kRecChunk; ++t)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float la2 = rate[j] * rec_sigmoid<kExact>(r[t].get(j));
                a[t][j] = exp2_fast(la2);
                const float m = __builtin_amdgcn_sqrtf(rec_keep2<kExact>(la2, a[t][j]));
                b[t][j] = m * rec_sigmoid<kExact>(i[t].get(j)) * x[t].get(j);
                H[j] = __builtin_fmaf(a[t][j], H[j], b[t][j]);
                A[j] *= a[t][j];
            }
        if (c.live)
#pragma unroll
            for (int j = 0; j < C; ++j) agg[slot + j] = make_float2(A[j], H[j]);
    }
    __syncthreads();
    join_chunks<T, C, MULTI, false>(p, agg, at, base_row, blocks_of_row);
    __syncthreads();
    if (!c.live || c.n <= 0) return;
    float h[C];
#pragma unroll
    for (int j = 0; j < C; ++j) h[j] = agg[slot + j].x;
    T* y = static_cast<T*>(p.y) + c.tok * p.D + c.ch;
#pragma unroll
    for (int t = 0; t < kRecChunk; ++t, y += p.D) {
#pragma unroll
        for (int j = 0; j < C; ++j) h[j] = __builtin_fmaf(a[t][j], h[j], b[t][j]);
        if (t < c.n) RecPack<T, C>::store(y, h);
    }
}

template <typename T, int C, bool MULTI>
__global__ __launch_bounds__(kThreads, 4) void rec_bwd_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    __shared__ float2 agg[kThreads * C];
    __shared__ uint32_t shared[2];
    RecPlace at;
    int64_t base_row;
    int blocks_of_row, slot;
    Chunk c;
    bool row_start;
    if (!lane_place<T, C, MULTI, true>(p, shared, at, base_row, blocks_of_row, c, slot, row_start)) return;
    const RecPlan& q = p.plan;
    RecPack<T, C> r[kRecChunk], g[kRecChunk], i[kRecChunk], x[kRecChunk], y[kRecChunk];
    load_chunk<T, C>(r, p.r, p.ldr, c, RecPack<T, C>::kMinusInf);
    load_chunk<T, C>(g, p.dy, p.D, c, 0);
    load_chunk<T, C>(i, p.i, p.ldi, c, 0);
    load_chunk<T, C>(x, p.x, p.ldx, c, 0);
    {  // the states before the tokens: the outputs one earlier
        const T* w = static_cast<const T*>(p.y) + (c.tok - 1) * p.D + c.ch;
#pragma unroll
        for (int t = 0; t < kRecChunk; ++t, w += p.D) {
            y[t].v = 0;
            if (c.live && t < c.n && !(t == 0 && row_start)) y[t].load(w);
        }
    }
    float rate[C], h0[C], u[C];
    {
        float A[C], U[C];
        const int64_t s = base_row + (MULTI ? 0 : (int)threadIdx.x / (q.nc * q.nt));
#pragma unroll
        for (int j = 0; j < C; ++j) {
            rate[j] = c.live ? rec_rate(p.lam[c.ch + j], p.c) : 0.0f;
            h0[j] = p.h0 && c.live && row_start && c.n > 0 ? p.h0[s * p.D + c.ch + j] : 0.0f;
            A[j] = 1.0f, U[j] = 0.0f;
        }
#pragma unroll
        for (int t = kRecChunk - 1; t >= 0; --t)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float a = exp2_fast(rate[j] * rec_sigmoid<kExact>(r[t].get(j)));
                U[j] = a * (U[j] + g[t].get(j));
                A[j] *= a;
            }
        if (c.live)
#pragma unroll
            for (int j = 0; j < C; ++j) agg[slot + j] = make_float2(A[j], U[j]);
    }
    __syncthreads();
    join_chunks<T, C, MULTI, true>(p, agg, at, base_row, blocks_of_row);
    __syncthreads();
    float sum[C];
#pragma unroll
    for (int j = 0; j < C; ++j) sum[j] = 0.0f, u[j] = c.live ? agg[slot + j].x : 0.0f;
    __syncthreads();
    if (c.live) {
#pragma unroll
        for (int t = kRecChunk - 1; t >= 0; --t) {
            if (t >= c.n) continue;
            float dx[C], dr[C], di[C];
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float sr = rec_sigmoid<kExact>(r[t].get(j)), si = rec_sigmoid<kExact>(i[t].get(j));
                const float la2 = rate[j] * sr, a = exp2_fast(la2), em = rec_keep2<kExact>(la2, a);
                const float rs = em > 0.0f ? __builtin_amdgcn_rsqf(em) : em == em ? 0.0f : em;
                const float G = g[t].get(j) + u[j], xv = x[t].get(j);
                const float before = t == 0 && row_start ? h0[j] : y[t].get(j);
                const float P = G * (a * (la2 * kLn2)) * (before - a * rs * si * xv);
                dx[j] = G * (em * rs) * si;
                di[j] = dx[j] * xv * (1.0f - si);
                dr[j] = P * (1.0f - sr);
                sum[j] += P;
                u[j] = a * G;
            }
            const int64_t o = (c.tok + t) * p.D + c.ch;
            RecPack<T, C>::store(static_cast<T*>(p.dx) + o, dx);
            RecPack<T, C>::store(static_cast<T*>(p.dr) + o, dr);
            RecPack<T, C>::store(static_cast<T*>(p.di) + o, di);
        }
        float* part = reinterpret_cast<float*>(agg) + slot;
#pragma unroll
        for (int j = 0; j < C; ++j) part[j] = sum[j];
    }
    __syncthreads();
    const int width = q.nc * C;
    for (int m = threadIdx.x; m < width; m += blockDim.x) {
        const int ch = at.tile * width + m;
        if (ch >= p.D) continue;
        const float* part = reinterpret_cast<const float*>(agg) + m;
        float all = 0.0f;
        for (int k = 0; k < q.nr * q.nt; ++k) all += part[k * width];
        p.w_lam[at.entry * p.D + ch] = all;
    }
}

// dlam from the workgroups' parts: 32 channels to a workgroup, every 32nd part to a lane.  softplus(lam) ->
// sigmoid(lam) (1 + e^lam / 2) as lam falls: their quotient is 1 in float32 below -17.
__global__ __launch_bounds__(1024) void rec_lam_kernel(const RecParams p) {
    __shared__ double part[32][33];
    const int w = threadIdx.x & 31, g = threadIdx.x >> 5, d = blockIdx.x * 32 + w;
    double sum = 0.0;
    if (d < p.D)
        for (int64_t k = g; k < p.plan.entries; k += 32) sum += (double)p.w_lam[k * p.D + d];
    part[g][w] = sum;
    __syncthreads();
    if (g || d >= p.D) return;
    for (int k = 1; k < 32; ++k) sum += part[k][w];
    const float lam = p.lam[d];
    const float ratio = lam < -17.0f ? 1.0f : rec_sigmoid<true>(lam) / (softplus_log2e(lam) * kLn2);
    p.dlam[d] = (float)sum * ratio;
}

// Tickets and words to all ones.
__global__ __launch_bounds__(256) void rec_clear_kernel(uint4* w, int64_t n) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k < n) w[k] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

template <typename T>
__global__ __launch_bounds__(256) void rec_step_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    const int d = blockIdx.y * 256 + threadIdx.x, s = blockIdx.x;
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

template <typename T, bool BACK>
hipError_t launch_rows(const RecParams& p, hipStream_t s) {
    constexpr int W = sizeof(T) == 4 ? 1 : 2;
    const RecPlan& q = p.plan;
    if (q.multi) {
        const int64_t n = q.bytes_words / 16;
        hipLaunchKernelGGL(rec_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, reinterpret_cast<uint4*>(p.w_tickets), n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)q.launch), threads((unsigned)(q.nr * q.nt * q.nc));
#define SFM_REC_LAUNCH(C, M)                                                                   \
    if (q.lane == C && q.multi == M) {                                                         \
        if constexpr (BACK)                                                                    \
            hipLaunchKernelGGL((rec_bwd_kernel<T, C, M>), grid, threads, 0, s, p);             \
        else                                                                                   \
            hipLaunchKernelGGL((rec_fwd_kernel<T, C, M>), grid, threads, 0, s, p);             \
    }
    SFM_REC_LAUNCH(1, 0) SFM_REC_LAUNCH(1, 1)
    if constexpr (W == 2) { SFM_REC_LAUNCH(2, 0) SFM_REC_LAUNCH(2, 1) }
#undef SFM_REC_LAUNCH
    return hipGetLastError();
}

}  // namespace

RecPlan plan_rec(int64_t rows, int64_t L, int64_t tokens, int64_t D, bool packed, int lane, bool back) {
    RecPlan q{};
    q.lane = lane;
    const int lanes = (int)((D + lane - 1) / lane);
    const int64_t chunks = (L + kRecChunk - 1) / kRecChunk;
    const int least = lanes < 32 ? lanes : 32;  // lanes side by side: 128 bytes where there are so many
    const int most = kThreads / (least < 16 ? least : 16) < 64 ? kThreads / (least < 16 ? least : 16) : 64;
    q.multi = chunks > most;
    q.nt = q.multi ? (kThreads / least < 64 ? kThreads / least : 64) : (int)chunks;
    // one block: as wide as the workgroup allows in whole 128 bytes, down to half that where it leaves fewer lanes idle
    int nc = q.multi ? least : kThreads / q.nt;
    if (nc >= lanes) {
        nc = lanes;
    } else if (nc >= 32) {
        const int widest = nc / 32 * 32;
        nc = widest;
        for (int n = widest - 32; n >= 32 && 2 * n >= widest; n -= 32)
            if ((lanes + n - 1) / n * n < (lanes + nc - 1) / nc * nc) nc = n;
    }
    q.nc = nc;
    q.tiles = (lanes + nc - 1) / nc;
    q.nr = q.multi || q.tiles > 1 ? 1 : kThreads / (q.nt * nc);
    if (q.nr > rows) q.nr = (int)rows;
    q.blocks = 1, q.groups = 1;
    const int64_t block = (int64_t)q.nt * kRecChunk;
    if (!q.multi) {
        q.entries = (rows + q.nr - 1) / q.nr;
        q.launch = q.entries * q.tiles;
    } else if (packed) {
        q.entries = tokens / block + rows;
        q.launch = q.entries * q.tiles;
    } else {
        q.blocks = (int)((L + block - 1) / block);
        q.groups = rows < 8 ? (int)rows : 8;
        q.entries = rows * q.blocks;
        q.launch = (rows + q.groups - 1) / q.groups * q.groups * q.blocks * q.tiles;
    }
    q.bytes_words = q.multi ? (int64_t)q.tiles * q.groups * 64 + q.entries * q.tiles * nc * lane * 8 : 0;
    q.bytes_words = (q.bytes_words + 15) / 16 * 16;
    q.bytes = q.bytes_words + (back ? q.entries * D * 4 : 0);
    return q;
}

hipError_t launch_rec_fwd(const RecParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_rows<float, false>(p, s) : launch_rows<__bf16, false>(p, s);
}

hipError_t launch_rec_bwd(const RecParams& p, int io_dtype, hipStream_t s) {
    const hipError_t e = io_dtype == 0 ? launch_rows<float, true>(p, s) : launch_rows<__bf16, true>(p, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(rec_lam_kernel, dim3((unsigned)((p.D + 31) / 32)), dim3(1024), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_rec_step(const RecParams& p, int io_dtype, hipStream_t s) {
    const dim3 grid((unsigned)p.rows, (unsigned)((p.D + 255) / 256));
    if (io_dtype == 0)
        hipLaunchKernelGGL(rec_step_kernel<float>, grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL(rec_step_kernel<__bf16>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
