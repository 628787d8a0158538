// delta_chunk.h -- the gated delta rule by chunks of 64 tokens (gfx950): what its forward and backward share.
//
// With G the running sum of the log decays inside a chunk, D_ij = exp(G_i - G_j) for j <= i, S0 the state before
// the chunk, and (rows are tokens)
//     M = strictly lower part of beta_i D_ij k_i.k_j,     T = (I + M)^-1,
//     R = beta (V - e^G K S0),   U = T R,   A = scale x lower part of D_ij q_i.k_j,
// the recurrence gives    O = scale e^G Q S0 + A U,     S' = e^(G_C) S0 + (e^(G_C - G) K)^T U.
// Every D_ij is at most one (g <= 0): it is e^(G_i) e^(-G_j) where a chunk's factors are within 2^-64 .. 2^64, and
// otherwise an exponential of its own, so nothing overflows.  Query and key lengths (l2norm), decays and gates
// are factors of whole rows or columns: they are applied to float32 accumulators, and the input operands of the
// matrix instructions stay the tensors' own values.
//
// LDS holds a chunk's K and Q (tokens x keys; the state's update reads K transposed), M, then T and A as computed
// operands (delta_mma.h).  Row pitches are an odd number of 16-byte units, so the sixteen rows of a fragment lie on
// different banks.
#pragma once

#include "delta_mma.h"
#include "sfm_delta.h"

namespace sfm {

constexpr int kC = kDeltaChunk;
constexpr int kDeltaThreads = 256;

// Row scalars of a chunk, in LDS.
struct ChunkRows {
    float ghi[kC], glo[kC];  // running sum of g log2(e) in two parts: differences of near values are exact
    float eg[kC];            // e^G
    float em[kC];            // e^-G where all of the chunk's e^G lie within 2^-64 .. 2^64, else zeros
    float er[kC];            // e^(G_C - G)
    float beta[kC];
    float rk[kC], rq[kC];    // 1 / length of the key and of the query (1 without l2norm)
};

template <typename T, int DK> struct ChunkShape {
    static constexpr int KS = DK + 16 / (int)sizeof(T);  // pitch of [token][key] arrays
    static constexpr int row_bytes = kC * KS * (int)sizeof(T);
};
// M in float32: ten lower tiles, each [column][row] (transposed), pitch 20
constexpr int kTileM = 16 * 20;
constexpr int kBytesM = 10 * kTileM * 4;
__device__ __forceinline__ constexpr int tile_at(int ti, int tj) { return (ti * (ti + 1) / 2 + tj) * kTileM; }

// Sum over the 8 or 16 lanes that hold a row (neighbours), by lane exchanges inside the vector unit.
template <int CTRL> __device__ __forceinline__ float dpp_get(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
    v += dpp_get<0xB1>(v);   // lanes 1, 0, 3, 2
    v += dpp_get<0x4E>(v);   // lanes 2, 3, 0, 1
    v += dpp_get<0x141>(v);  // mirror of eight
    if (LANES == 16) v += dpp_get<0x140>(v);  // mirror of sixteen
    return v;
}
// a float64 from the lanes below: CTRL of the wave's scan, zero where there is none
template <int CTRL, int ROWS> __device__ __forceinline__ double dpp_below(double v) {
    const long long b = __builtin_bit_cast(long long, v);
    const int lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, false);
    return __builtin_bit_cast(double, (long long)(((unsigned long long)(unsigned)hi << 32) | (unsigned)lo));
}

// this thread's number among the 256 that share a chunk's loads
__device__ __forceinline__ unsigned share_id() { return threadIdx.x & (kDeltaThreads - 1); }

// One thread's share of a chunk's [64][DK] rows: eight keys of every 2048 / DK-th token.
template <typename T, int DK> struct RowShare {
    static constexpr int kPer = DK / 8, kUnits = kC * kPer / kDeltaThreads, kStep = kDeltaThreads / kPer;
    typedef T vec8 __attribute__((ext_vector_type(8)));
    vec8 a[kUnits];

    // the buffer holds the chunk's rows, ld apart, from the head's first key on; zeros behind its end and behind dk
    __device__ __forceinline__ void load(const Buf& b, int64_t ld, int dk, bool vec) {
        constexpr int per = 16 / (int)sizeof(T);
        typedef T piece __attribute__((ext_vector_type(per)));
        const int t0 = share_id() / kPer, c = share_id() % kPer * 8;
        const unsigned at = fresh((unsigned)(t0 * ld + c) * (unsigned)sizeof(T)), step = (unsigned)(kStep * ld) * (unsigned)sizeof(T);
        if (vec) {
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
#pragma unroll
                for (int j = 0; j < 8 / per; ++j) {
                    const piece x = buf_load<piece>(b, (c + j * per < dk ? at + j * 16u : kNowhere) + i * step);
#pragma unroll
                    for (int e = 0; e < per; ++e) a[i][j * per + e] = x[e];
                }
        } else {
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    a[i][e] = buf_load<T>(b, (c + e < dk ? at + e * (unsigned)sizeof(T) : kNowhere) + i * step);
        }
    }

    // into LDS: the rows and, if wanted, one over their lengths
    __device__ __forceinline__ void store(T* rows, float* factor, int l2norm) const {
        using Sh = ChunkShape<T, DK>;
        const int t0 = share_id() / kPer, c = share_id() % kPer * 8;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) *reinterpret_cast<vec8*>(rows + (t0 + i * kStep) * Sh::KS + c) = a[i];
        if (!factor) return;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            float f = 1.0f;
            if (l2norm) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = to_f32((T)a[i][e]);
                    s = __builtin_fmaf(x, x, s);
                }
                f = __builtin_amdgcn_rsqf(lanes_sum<kPer>(s) + kDeltaNormEps);
            }
            if (c == 0) factor[t0 + i * kStep] = f;
        }
    }
};

// Decays and gates of a chunk (one wave, a lane to a token; tokens past n: no decay, no gate).  The running sum is
// taken in float64 (its differences, not its values, are what counts).
struct ChunkGates {
    float g, beta;
    template <typename T> __device__ __forceinline__ void load(const T* gp, const T* bp, int64_t ld, int n) {
        const int lane = threadIdx.x & 63;
        const unsigned at = (unsigned)(lane * ld) * (unsigned)sizeof(T);
        g = Io<T>::of_bits(buf_load_bits<T>(make_buf(gp, n * ld * (int)sizeof(T)), at));
        beta = Io<T>::of_bits(buf_load_bits<T>(make_buf(bp, n * ld * (int)sizeof(T)), at));
    }
    __device__ __forceinline__ void store(ChunkRows* rows) const {
        const int lane = threadIdx.x & 63;
        double s = (double)(g < kDeltaMinGate ? kDeltaMinGate : g) * 1.4426950408889634;
        s += dpp_below<0x111, 0xf>(s);  // lanes 1, 2, 4, 8 below in the row of sixteen
        s += dpp_below<0x112, 0xf>(s);
        s += dpp_below<0x114, 0xf>(s);
        s += dpp_below<0x118, 0xf>(s);
        s += dpp_below<0x142, 0xa>(s);  // lane 15 of the row before, for rows 1 and 3
        s += dpp_below<0x143, 0xc>(s);  // lane 31, for rows 2 and 3
        const double end = __shfl(s, 63);
        const float hi = (float)s, lo = (float)(s - (double)hi);
        rows->ghi[lane] = hi;
        rows->glo[lane] = lo;
        // the sum's own rounding as a factor: both exponentials good to their last places, and so their products
        const float fix = lo * kLn2;
        const float e = exp2_fast(hi), m = exp2_fast(-hi);
        rows->eg[lane] = __builtin_fmaf(e, fix, e);
        rows->em[lane] = __ballot(fabsf(hi) <= 64.0f) == ~0ull ? __builtin_fmaf(-m, fix, m) : 0.0f;
        rows->er[lane] = exp2_fast((float)(end - s));
        rows->beta[lane] = beta;
    }
};

// Whether a decay between two tokens is the product e^(G_i) e^(-G_j): neither factor, nor its product with a row's,
// leaves float32's range.  Otherwise each pair takes an exponential of its own.
__device__ __forceinline__ bool mild_decay(const ChunkRows* rows) { return __builtin_amdgcn_readfirstlane(rows->em[0] > 0.0f); }

// tile number 0..9 of the lower triangle of 4 x 4 tiles -> its row and column
__device__ __forceinline__ void lower_tile(int n, int& ti, int& tj) {
    ti = n >= 6 ? 3 : (n >= 3 ? 2 : (n >= 1 ? 1 : 0));
    tj = n - ti * (ti + 1) / 2;
}

// four neighbouring row scalars
__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// c = rows of a (tile ta) times rows of b (tile tb), over all keys: lane l has a's rows 4 (l / 16) .. + 3, b's row l % 16
template <typename T, int DK> __device__ __forceinline__ f32x4 rows_product(const T* a, int ta, const T* b, int tb) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, at = (lane & 15) * Sh::KS + (lane >> 4) * 4;
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < DK; kb += 32)
        c = mma(load_runs<T>(a + ta * 16 * Sh::KS + at + kb), load_runs<T>(b + tb * 16 * Sh::KS + at + kb), c);
    return c;
}

// The twenty lower tiles of K K^T (for M) and Q K^T (for A), five to a wave: task w + 4 n, M's ten first.
template <typename T, int DK> __device__ __forceinline__ void chunk_products(const T* ks, const T* qs, f32x4 (&c)[5]) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int n = 0; n < 5; ++n) c[n] = f32x4{0, 0, 0, 0};
    constexpr int step = sizeof(T) == 4 ? 32 : 64;  // keys whose fragments are loaded together
#pragma unroll
    for (int k0 = 0; k0 < DK; k0 += step) {
        Frag<T> fa[5][step / 32], fb[5][step / 32];
#pragma unroll
        for (int n = 0; n < 5; ++n) {
            const int id = wave + 4 * n;
            const bool m = id < 10;
            int ti, tj;
            lower_tile(m ? id : id - 10, ti, tj);
            const int at = l16 * Sh::KS + g4 + k0;
#pragma unroll
            for (int i = 0; i < step / 32; ++i) {
                fa[n][i] = load_runs<T>(ks + (m ? ti : tj) * 16 * Sh::KS + at + i * 32);
                fb[n][i] = load_runs<T>((m ? ks : qs) + (m ? tj : ti) * 16 * Sh::KS + at + i * 32);
            }
        }
        loads_end();
#pragma unroll
        for (int i = 0; i < step / 32; ++i)
#pragma unroll
            for (int n = 0; n < 5; ++n) c[n] = mma(fa[n][i], fb[n][i], c[n]);
    }
}

// M and A from them and a head's gates.  M goes to LDS; A's tiles stay in registers (a[n - 2]; lane: row i = l % 16,
// columns 4 (l / 16) .. + 3) until M's place is free.
__device__ __forceinline__ void chunk_triangles(const f32x4 (&c)[5], const ChunkRows* rows, float scale, float* mt, f32x4 (&a)[3]) {
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
    const bool mild = mild_decay(rows);
#pragma unroll
    for (int n = 0; n < 5; ++n) {
        const int id = wave + 4 * n;
        int ti, tj;
        lower_tile(id < 10 ? id : id - 10, ti, tj);
        if (n < 2 || (n == 2 && id < 10)) {
            const int j = tj * 16 + l16, i0 = ti * 16 + g4;
            const f32x4 f = four(rows->rk + i0) * four(rows->beta + i0);
            f32x4 m;
            if (mild) {
                const float fj = rows->rk[j] * rows->em[j];
                m = c[n] * (f * four(rows->eg + i0) * fj);
            } else {
                const float fj = rows->rk[j], hj = rows->ghi[j], lj = rows->glo[j];
                const f32x4 hi = four(rows->ghi + i0), lo = four(rows->glo + i0);
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = i0 + r > j ? c[n][r] * fj * f[r] * exp2_fast((hi[r] - hj) + (lo[r] - lj)) : 0.0f;
            }
            if (ti == tj)
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = g4 + r > l16 ? m[r] : 0.0f;
            *reinterpret_cast<f32x4*>(mt + tile_at(ti, tj) + l16 * 20 + g4) = m;
        } else {
            const int i = ti * 16 + l16, j0 = tj * 16 + g4;
            const float fi = scale * rows->rq[i];
            f32x4& x = a[n < 2 ? 0 : n - 2];
            if (mild) {
                x = c[n] * (four(rows->rk + j0) * four(rows->em + j0) * (fi * rows->eg[i]));
            } else {
                const float hi = rows->ghi[i], lo = rows->glo[i];
                const f32x4 hj = four(rows->ghi + j0), lj = four(rows->glo + j0), rj = four(rows->rk + j0);
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = j0 + r <= i ? c[n][r] * (fi * rj[r]) * exp2_fast((hi - hj[r]) + (lo - lj[r])) : 0.0f;
            }
            if (ti == tj)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = g4 + r <= l16 ? x[r] : 0.0f;
        }
    }
}

// A's tiles (of chunk_products) one by one: f(tile, row tile, column tile), and zeros for the tile right of a diagonal
// one that shares its step of 32
template <typename F> __device__ __forceinline__ void each_a(const f32x4 (&a)[3], F f) {
    const int wave = wave_id();
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int id = wave + 4 * n - 2;  // task w + 4 (n + 2), less M's ten
        if (id < 0) continue;
        int ti, tj;
        lower_tile(id, ti, tj);
        f(a[n], ti, tj);
        if (ti == tj && !(ti & 1)) f(f32x4{0, 0, 0, 0}, ti, tj + 1);
    }
}

// Inverse of the unit lower triangular 16 x 16 block `wave` of I + M in M's place, kept transposed, [column][row]:
// column c by lane c (lanes repeat).  Column-oriented substitution: once x_k is known every later x_i takes its
// share, so the chain is 15 steps of independent operations.
__device__ __forceinline__ void invert_diagonal(float* mt) {
    const int lane = threadIdx.x & 63, wave = wave_id(), c = lane & 15;
    float* m = mt + tile_at(wave, wave);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < 15; ++k)
#pragma unroll
        for (int q = k / 4; q < 4; ++q) {
            const f32x4 col = four(m + k * 20 + q * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q * 4 + j > k) x[q * 4 + j] = __builtin_fmaf(-col[j], x[k], x[q * 4 + j]);
        }
    if (lane < 16) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(m + c * 20 + q * 4) = f32x4{x[q * 4], x[q * 4 + 1], x[q * 4 + 2], x[q * 4 + 3]};
    }
}

// Rows 16 wave .. + 15 of T from M with its diagonal blocks inverted, in float32 matrix instructions:
//     T_ij = -(sum over k = j + 1 .. i of T_ik M_kj) T_jj,   j = i - 1 .. 0,
// each block transposed, so a block is the next one's operand where it lies.  t[j]: lane has row l % 16 of the
// block, columns 4 (l / 16) .. + 3.
__device__ __forceinline__ void inverse_rows(const float* mt, f32x4 (&t)[4]) {
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
        t[j] = f32x4{0, 0, 0, 0};
        if (j == wave) {
#pragma unroll
            for (int r = 0; r < 4; ++r) t[j][r] = mt[tile_at(j, j) + (g4 + r) * 20 + l16];
        } else if (j < wave) {
            f32x4 z = {0, 0, 0, 0};
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (k > j && k <= wave) z = mma4(four(mt + tile_at(k, j) + l16 * 20 + g4), t[k], z);
            t[j] = mma4(-four(mt + tile_at(j, j) + l16 * 20 + g4), z, t[j]);
        }
    }
}

// T's tiles of this wave likewise
template <typename F> __device__ __forceinline__ void each_t(const f32x4 (&t)[4], F f) {
    const int wave = wave_id();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j <= (wave | 1)) f(t[j], wave, j);
}

// Gates, K and Q (in registers) to LDS, and their products.
template <typename T, int DK>
__device__ __forceinline__ void start_chunk(const RowShare<T, DK>& kr, const RowShare<T, DK>& qr, const ChunkGates& gates,
                                            const DeltaParams& p, ChunkRows* rows, T* ks, T* qs, f32x4 (&c)[5]) {
    if (wave_id() == 3) gates.store(rows);  // (its loads are the oldest; this wave has least to do below)
    kr.store(ks, rows->rk, p.l2norm);
    qr.store(qs, rows->rq, p.l2norm);
    lds_barrier();
    chunk_products<T, DK>(ks, qs, c);
}
// From them M in LDS and, in registers, A's tiles and this wave's rows of T, all by the whole workgroup.  `after` runs
// between M's making and its use (what needs K, Q or A only).
template <typename After>
__device__ __forceinline__ void finish_chunk(const f32x4 (&c)[5], const DeltaParams& p, const ChunkRows* rows, float* mt,
                                             f32x4 (&a)[3], f32x4 (&t)[4], After after) {
    chunk_triangles(c, rows, p.scale, mt, a);
    lds_barrier();
    after();
    invert_diagonal(mt);
    lds_barrier();
    inverse_rows(mt, t);
}

// Both, with T (PT parts) at ts and A (PA parts) at as, where M lies before, visible to all at the end.
template <typename T, int DK, int PT, int PA, typename After, typename Between>
__device__ __forceinline__ void build_chunk(const RowShare<T, DK>& kr, const RowShare<T, DK>& qr, const ChunkGates& gates,
                                            const DeltaParams& p, ChunkRows* rows, T* ks, T* qs, T* as, T* ts,
                                            After after, Between between) {
    f32x4 c[5], a[3], t[4];
    start_chunk<T, DK>(kr, qr, gates, p, rows, ks, qs, c);
    finish_chunk(c, p, rows, reinterpret_cast<float*>(as), a, t, after);
    each_t(t, [&](f32x4 x, int rt, int tj) { store_tile<PT>(x, ts, rt, tj); });
    between();     // what needs K and Q only
    lds_barrier();  // M is done with
    each_a(a, [&](f32x4 x, int rt, int tj) { store_tile<PA>(x, as, rt, tj); });
    lds_barrier();
}

// A row's place in the arrays that hold something for every chunk: chunk c of row s is entry first + c.  Packed
// rows: first = start / 64 + s leaves every row room for its chunks without a count of those before it.
__device__ __forceinline__ unsigned chunk_entry(const DeltaParams& p, int s, int64_t first) {
    return p.offsets ? (unsigned)(first / kC) + s : (unsigned)s * ((p.L + kC - 1) / kC);
}

// The chunk that an entry holds, for the kernels that take the entries one by one: its row, that row's first token and
// length, and where in the row it starts.  Packed rows: the last row whose first entry is not past this one, found by
// the wave 64 rows at a time (one step to 64 rows, two to 4096).
struct ChunkAt {
    int s, len;
    int64_t first, t0;
};
__device__ __forceinline__ bool chunk_at(const DeltaParams& p, unsigned entry, ChunkAt& at) {
    if (!p.offsets) {
        const unsigned chunks = (unsigned)(p.L + kC - 1) / kC;
        at.s = (int)(entry / chunks);
        delta_row(p, at.s, at.first, at.len);
        at.t0 = (int64_t)(entry - (unsigned)at.s * chunks) * kC;
        return at.t0 < at.len;
    }
    int lo = 0, n = p.rows;
    for (;;) {
        const int step = (n + 63) / 64, i = (threadIdx.x & 63) * step;
        bool before = false;
        if (i < n) {
            const int64_t o = p.offsets[lo + i], first = o < 0 ? 0 : o > p.tokens ? p.tokens : o;
            before = (unsigned)(first / kC) + (unsigned)(lo + i) <= entry;
        }
        const int there = __builtin_popcountll(__ballot(before));
        if (there == 0) return false;  // (tokens before the first row)
        const int at_lane = (there - 1) * step;
        lo += at_lane;
        n = min(step, n - at_lane);
        if (step == 1) break;
    }
    at.s = lo;
    delta_row(p, at.s, at.first, at.len);
    at.t0 = ((int64_t)entry - (int64_t)chunk_entry(p, at.s, at.first)) * kC;
    return at.t0 >= 0 && at.t0 < at.len;  // (a row leaves up to one entry free)
}

// What the preparing kernel leaves of a chunk and head: the row scalars, T and A (P parts each).
template <typename T, int P, int PA = P> struct ChunkOperands {
    static constexpr int frag_bytes = kLowerFrags * kFragSize * (int)sizeof(T);
    static constexpr int t = (int)sizeof(ChunkRows), a = t + P * frag_bytes, bytes = a + PA * frag_bytes;
    static_assert(sizeof(ChunkRows) % 16 == 0 && frag_bytes % 16 == 0, "whole 16-byte units");
};

// One thread's share of such a run of 16-byte units, N bytes long
template <int N> struct Linear {
    typedef unsigned unit __attribute__((ext_vector_type(4)));
    static constexpr int kUnits = (N / 16 + kDeltaThreads - 1) / kDeltaThreads;
    unit x[kUnits];
    __device__ __forceinline__ void load(const char* p, bool there = true) {
        const Buf b = make_buf(p, there ? N : 0);
#pragma unroll
        for (int i = 0; i < kUnits; ++i) x[i] = buf_load<unit>(b, (share_id() + i * kDeltaThreads) * 16u);
    }
    __device__ __forceinline__ void store(char* p) const {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = share_id() + i * kDeltaThreads;
            if (N % (kDeltaThreads * 16) == 0 || u < N / 16) *reinterpret_cast<unit*>(p + u * 16) = x[i];
        }
    }
};

// Workgroup -> unit of work: workgroups go to the eight dies in turn.  Runs of `run` neighbouring units stay on one
// die, so its L2 serves what they share, and the runs go to the dies in turn.
__device__ __forceinline__ unsigned die_local(unsigned id, unsigned n, unsigned run) {
    const unsigned whole = n / (8 * run) * (8 * run);
    if (id < whole) {
        const unsigned die = id % 8, at = id / 8, r = at / run;
        return (r * 8 + die) * run + (at - r * run);
    }
    n -= whole, id -= whole;  // fewer than eight runs: a stretch to each
    const unsigned per = n / 8, rest = n % 8, die = id % 8, at = id / 8;
    return whole + die * per + (die < rest ? die : rest) + at;
}

// The same with `row` units to a row, `keys` of them reading the same keys.  Equal rows: a row's all go to one die, in
// every kernel, whose L2 then holds what one kernel leaves the next.  Rows that differ in length, or too few for that:
// only what reads the same keys, so that long rows weigh on all dies alike (24 packed rows: 166 us, 184 with an eighth
// of the rows to each die; backward of 2 rows x 4002 tokens: 246 us, 252).
__device__ __forceinline__ unsigned row_unit(const DeltaParams& p, unsigned id, unsigned n, unsigned row, unsigned keys) {
    return die_local(id, n, p.offsets || p.rows < 8 ? keys : row);
}

}  // namespace sfm
