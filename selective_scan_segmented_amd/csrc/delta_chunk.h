// delta_chunk.h -- the gated delta rule by chunks of 64 tokens (gfx950): what its forward and backward share.
//
// With G the running sum of the log decays inside a chunk, D_ij = exp(G_i - G_j) for j <= i, S0 the state before
// the chunk, and (rows are tokens)
//     M = strictly lower part of beta_i D_ij k_i.k_j,     T = (I + M)^-1,
//     R = beta (V - e^G K S0),   U = T R,   A = scale x lower part of D_ij q_i.k_j,
// the recurrence gives    O = scale e^G Q S0 + A U,     S' = e^(G_C) S0 + (e^(G_C - G) K)^T U.
// Every exponent is at most zero (g <= 0), so nothing overflows.  Query and key lengths (l2norm), decays and gates
// are factors of whole rows or columns: they are applied to float32 accumulators, and the input operands of the
// matrix instructions stay the tensors' own values.
//
// LDS holds a chunk's K and Q (tokens x keys), K again the other way round (keys x tokens, for the state's
// update), M, then T and A as computed operands (delta_mma.h).  Row pitches are an odd number of 16-byte units, so
// the sixteen rows of a fragment lie on different banks.
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
    float er[kC];            // e^(G_C - G)
    float beta[kC];
    float rk[kC], rq[kC];    // 1 / key length; scale / query length
};

template <typename T, int DK> struct ChunkShape {
    static constexpr int kPad = 16 / (int)sizeof(T);
    static constexpr int KS = DK + kPad;   // pitch of [token][key] arrays
    static constexpr int TS = kC + kPad;   // pitch of [..][token] arrays
    static constexpr int MS = kC + 4;      // pitch of the float32 M
};

// Eight neighbouring elements of a row, zeros from element n on.
template <typename T> struct Raw8 {
    typedef T vec __attribute__((ext_vector_type(8)));
    vec v;
};
template <typename T> __device__ __forceinline__ Raw8<T> load8(const T* p, int n, bool vec) {
    constexpr int per = 16 / (int)sizeof(T);
    typedef T piece __attribute__((ext_vector_type(per)));
    Raw8<T> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = Io<T>::zero();
    if (vec) {
#pragma unroll
        for (int i = 0; i < 8 / per; ++i)
            if (n > i * per) {
                const piece x = *reinterpret_cast<const piece*>(p + i * per);
#pragma unroll
                for (int e = 0; e < per; ++e) r.v[i * per + e] = x[e];
            }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) r.v[e] = p[e];
    }
    return r;
}
template <typename T> __device__ __forceinline__ T elem8(const Raw8<T>& r, int i) { return r.v[i]; }

// One thread's share of a chunk's [64][DK] rows: pairs of neighbouring tokens, eight keys each.
template <typename T, int DK> struct RowPairs {
    static constexpr int kUnits = kC / 2 * (DK / 8) / kDeltaThreads;
    Raw8<T> a[kUnits], b[kUnits];

    // rows: first valid row at p, stride ld; n of them exist
    __device__ __forceinline__ void load(const T* p, int64_t ld, int n, int dk, bool vec) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = threadIdx.x + i * kDeltaThreads, t = u / (DK / 8) * 2, c = u % (DK / 8) * 8;
            const T* at = p + t * ld + c;
            a[i] = load8<T>(at, t < n ? dk - c : 0, vec);
            b[i] = load8<T>(at + ld, t + 1 < n ? dk - c : 0, vec);
        }
    }

    // into LDS: rows [token][slot of key], the transpose [key][slot of token] if wanted, and the rows' factors
    __device__ __forceinline__ void store(T* rows, T* trans, float* factor, float scale, int l2norm) const {
        using Sh = ChunkShape<T, DK>;
        typedef T pair_t __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = threadIdx.x + i * kDeltaThreads, t = u / (DK / 8) * 2, c = u % (DK / 8) * 8;
            T* r0 = rows + t * Sh::KS;
            const int s0 = slot_of(c), s1 = slot_of(c + 4);
            copy4(r0 + s0, a[i], 0);
            copy4(r0 + s1, a[i], 4);
            copy4(r0 + Sh::KS + s0, b[i], 0);
            copy4(r0 + Sh::KS + s1, b[i], 4);
            if (trans) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    *reinterpret_cast<pair_t*>(trans + (c + e) * Sh::TS + slot_of(t)) =
                        pair_t{elem8<T>(a[i], e), elem8<T>(b[i], e)};
            }
            float sa = 0.0f, sb = 0.0f;
            if (l2norm) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = to_f32(elem8<T>(a[i], e)), y = to_f32(elem8<T>(b[i], e));
                    sa = __builtin_fmaf(x, x, sa);
                    sb = __builtin_fmaf(y, y, sb);
                }
#pragma unroll
                for (int m = 1; m < DK / 8; m <<= 1) {
                    sa += __shfl_xor(sa, m);
                    sb += __shfl_xor(sb, m);
                }
                sa = 1.0f / __builtin_sqrtf(sa + kDeltaNormEps);
                sb = 1.0f / __builtin_sqrtf(sb + kDeltaNormEps);
            } else {
                sa = sb = 1.0f;
            }
            if (c == 0) {
                factor[t] = scale * sa;
                factor[t + 1] = scale * sb;
            }
        }
    }

    static __device__ __forceinline__ void copy4(T* to, const Raw8<T>& r, int from) {
        typedef T quad_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<quad_t*>(to) =
            quad_t{elem8<T>(r, from), elem8<T>(r, from + 1), elem8<T>(r, from + 2), elem8<T>(r, from + 3)};
    }
};

// Decays and gates of a chunk (one wave, a lane to a token; tokens past n: no decay, no gate).  The running sum is
// taken in float64 (its differences, not its values, are what counts).
template <typename T>
__device__ __forceinline__ void chunk_gates(const T* g, const T* beta, int64_t ld, int n, ChunkRows* rows) {
    const int lane = threadIdx.x & 63;
    float gv = 0.0f, bv = 0.0f;
    if (lane < n) {
        gv = to_f32(g[lane * ld]);
        bv = to_f32(beta[lane * ld]);
        gv = gv < kDeltaMinGate ? kDeltaMinGate : gv;
    }
    double s = (double)gv * 1.4426950408889634;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const double o = __shfl_up(s, m);
        if (lane >= m) s += o;
    }
    const double end = __shfl(s, 63);
    const float hi = (float)s;
    rows->ghi[lane] = hi;
    rows->glo[lane] = (float)(s - (double)hi);
    rows->eg[lane] = exp2_fast((float)s);
    rows->er[lane] = exp2_fast((float)(end - s));
    rows->beta[lane] = bv;
}

__device__ __forceinline__ float decay(const ChunkRows* r, float hi, float lo, int j) {
    return exp2_fast((hi - r->ghi[j]) + (lo - r->glo[j]));
}

// tile number 0..9 of the lower triangle of 4 x 4 tiles -> its row and column
__device__ __forceinline__ void lower_tile(int n, int& ti, int& tj) {
    ti = n >= 6 ? 3 : (n >= 3 ? 2 : (n >= 1 ? 1 : 0));
    tj = n - ti * (ti + 1) / 2;
}

// c = rows of a (tile ta) times rows of b (tile tb), over all keys: lane l has a's rows 4 (l / 16) .. + 3, b's row l % 16
template <typename T, int DK> __device__ __forceinline__ f32x4 rows_product(const T* a, int ta, const T* b, int tb) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, at = (lane & 15) * Sh::KS + (lane >> 4) * 8;
    f32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int kb = 0; kb < DK; kb += 32)
        c = mma(Frag<T>::load(a + ta * 16 * Sh::KS + at + kb), Frag<T>::load(b + tb * 16 * Sh::KS + at + kb), c);
    return c;
}

// The lower tiles of M (transposed: mt[j][i]) and, in registers, of A (lane: row i = l % 16, columns 4 (l / 16) .. + 3;
// wave w holds tiles 3 - w, 7 - w and, if below 10, 11 - w).
template <typename T, int DK, bool WITH_A>
__device__ __forceinline__ void chunk_products(const T* ks, const T* qs, const ChunkRows* rows, float* mt, f32x4 (&a)[3]) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int id = wave + 4 * n;
        if (id >= 10) continue;
        int ti, tj;
        lower_tile(id, ti, tj);
        const f32x4 c = rows_product<T, DK>(ks, ti, ks, tj);
        const int j = tj * 16 + l16, i0 = ti * 16 + g4;
        const float rj = rows->rk[j], hj = rows->ghi[j], lj = rows->glo[j];
        f32x4 m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r;
            const float d = exp2_fast((rows->ghi[i] - hj) + (rows->glo[i] - lj));
            m[r] = i > j ? c[r] * (rows->rk[i] * rj) * (rows->beta[i] * d) : 0.0f;
        }
        *reinterpret_cast<f32x4*>(mt + j * Sh::MS + i0) = m;
    }
    if (WITH_A) {
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            const int id = 3 - wave + 4 * n;
            if (id >= 10) continue;
            int ti, tj;
            lower_tile(id, ti, tj);
            const f32x4 c = rows_product<T, DK>(ks, tj, qs, ti);
            const int i = ti * 16 + l16, j0 = tj * 16 + g4;
            const float ri = rows->rq[i], hi = rows->ghi[i], lo = rows->glo[i];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = j0 + r;
                a[n][r] = j <= i ? c[r] * (ri * rows->rk[j]) * decay(rows, hi, lo, j) : 0.0f;
            }
        }
    }
}

// A's tiles (of chunk_products) as a computed operand [row][slot of column]; tiles right of the diagonal that
// share a step of 32 with one on it are zeros.
template <typename T, int DK, int PA> __device__ __forceinline__ void store_a(const f32x4 (&a)[3], T* as) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const int id = 3 - wave + 4 * n;
        if (id >= 10) continue;
        int ti, tj;
        lower_tile(id, ti, tj);
        T* row = as + (ti * 16 + l16) * Sh::TS;
        store_parts<PA>(a[n], row + slot_of(tj * 16 + g4), kC * Sh::TS);
        if (ti == tj && !(ti & 1)) store_parts<PA>(f32x4{0, 0, 0, 0}, row + slot_of(tj * 16 + 16 + g4), kC * Sh::TS);
    }
}

// Inverse of the unit lower triangular 16 x 16 block `wave` of I + M: column c by lane c (lanes repeat), kept
// transposed, td[c][i].  Column-oriented substitution: once x_k is known every later x_i takes its share, so the
// chain is 15 steps of independent operations.
__device__ __forceinline__ void invert_diagonal(const float* mt, int ms, float* td) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15;
    const float* m = mt + wave * 16 * ms + wave * 16;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == c ? 1.0f : 0.0f;
#pragma unroll
    for (int k = 0; k < 15; ++k) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q * 4 + 3 <= k) continue;
            const f32x4 col = *reinterpret_cast<const f32x4*>(m + k * ms + q * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (q * 4 + j > k) x[q * 4 + j] = __builtin_fmaf(-col[j], x[k], x[q * 4 + j]);
        }
    }
    if (lane < 16) {
        float* out = td + wave * 16 * 20 + c * 20;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(out + q * 4) = f32x4{x[q * 4], x[q * 4 + 1], x[q * 4 + 2], x[q * 4 + 3]};
    }
}

// Rows 16 wave .. + 15 of T from the diagonal inverses, in float32 matrix instructions:
//     T_ij = -(sum over k = j + 1 .. i of T_ik M_kj) T_jj,   j = i - 1 .. 0,
// each block transposed, so a block is the next one's operand where it lies.  t[j]: lane has row l % 16 of the
// block, columns 4 (l / 16) .. + 3.
__device__ __forceinline__ void inverse_rows(const float* mt, int ms, const float* td, f32x4 (&t)[4]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
        t[j] = f32x4{0, 0, 0, 0};
        if (j == wave) {
#pragma unroll
            for (int r = 0; r < 4; ++r) t[j][r] = td[j * 320 + (g4 + r) * 20 + l16];
        } else if (j < wave) {
            f32x4 z = {0, 0, 0, 0};
#pragma unroll
            for (int k = 1; k < 4; ++k)
                if (k > j && k <= wave)
                    z = mma4(*reinterpret_cast<const f32x4*>(mt + (j * 16 + l16) * ms + k * 16 + g4), t[k], z);
            const f32x4 d = *reinterpret_cast<const f32x4*>(td + j * 320 + l16 * 20 + g4);
            t[j] = mma4(-d, z, t[j]);
        }
    }
}

// T's rows of this wave as a computed operand [row][slot of column]
template <typename T, int DK, int PT> __device__ __forceinline__ void store_t(const f32x4 (&t)[4], T* ts) {
    using Sh = ChunkShape<T, DK>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j <= (wave | 1)) store_parts<PT>(t[j], ts + (wave * 16 + l16) * Sh::TS + slot_of(j * 16 + g4), kC * Sh::TS);
}

// four neighbouring row scalars
__device__ __forceinline__ f32x4 four(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// Workgroup -> unit of work: workgroups go to the eight dies in turn, and neighbouring units (the column tiles and
// heads that read the same keys) stay on one die, so its L2 serves them.
__device__ __forceinline__ int64_t die_local(int64_t id, int64_t n) {
    const int64_t per = n / 8, rest = n % 8, die = id % 8, at = id / 8;
    return die * per + (die < rest ? die : rest) + at;
}

}  // namespace sfm
