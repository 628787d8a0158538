// delta_fwd.h -- the chunked forward of the gated delta rule (kernels; one translation unit per io type).
#pragma once

#include "delta_chunk.h"

namespace sfm {

// LDS of the forward, in bytes from the start.
template <typename T, int DK, int PS> struct FwdLds {
    using Sh = ChunkShape<T, DK>;
    static constexpr int PT = PS;                                  // parts of T
    static constexpr int PA = sizeof(T) == 4 ? 1 : 2;              // parts of A
    static constexpr int rows = 0;
    static constexpr int ks = (int)sizeof(ChunkRows);
    static constexpr int qs = ks + kC * Sh::KS * (int)sizeof(T);
    static constexpr int kt = qs + kC * Sh::KS * (int)sizeof(T);
    static constexpr int as = kt + DK * Sh::TS * (int)sizeof(T);   // A; M before it
    static constexpr int a_bytes = PA * kC * Sh::TS * (int)sizeof(T), m_bytes = kC * Sh::MS * 4;
    static constexpr int ts = as + (a_bytes > m_bytes ? a_bytes : m_bytes);
    static constexpr int td = ts + PT * kC * Sh::TS * (int)sizeof(T);
    static constexpr int bytes = td + 4 * 16 * 20 * 4;
};

// A workgroup takes one (row, head) and 64 NC columns of its values, NC tiles of 16 to a wave, and walks the
// row's chunks; the state's columns stay in the wave's accumulators (float32) all the way.
template <typename T, int DK, int NC, int PS>
__global__ __launch_bounds__(kDeltaThreads) void delta_fwd_kernel(const DeltaParams p, int tiles, int64_t units) {
    using Sh = ChunkShape<T, DK>;
    using L = FwdLds<T, DK, PS>;
    constexpr int PA = L::PA, PT = L::PT, PY = PS < 2 ? PS : 2;
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs),
      *kt = reinterpret_cast<T*>(lds + L::kt), *as = reinterpret_cast<T*>(lds + L::as),
      *ts = reinterpret_cast<T*>(lds + L::ts);
    float *mt = reinterpret_cast<float*>(lds + L::as), *td = reinterpret_cast<float*>(lds + L::td);

    const int64_t unit = die_local(blockIdx.x, units);
    const int64_t rh = unit / tiles;
    const int s = (int)(rh / p.H), h = (int)(rh - (int64_t)s * p.H), hk = h / (p.H / p.Hk);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int col0 = (int)(unit - rh * tiles) * 64 * NC + wave * 16 * NC + l16;
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
    const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
    const T* vp = static_cast<const T*>(p.v) + first * p.ldv + (int64_t)h * p.dv;
    const T* gp = static_cast<const T*>(p.g) + first * p.H + h;
    const T* bp = static_cast<const T*>(p.beta) + first * p.H + h;
    T* op = static_cast<T*>(p.o) + (first * p.H + h) * p.dv;
    const int64_t sbase = rh * p.dk * (int64_t)p.dv;

    f32x4 S[DK / 16][NC];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = d * 16 + g4 + r, c = col0 + n * 16;
                S[d][n][r] = p.h0 && row < p.dk && c < p.dv ? p.h0[sbase + (int64_t)row * p.dv + c] : 0.0f;
            }
    bool zero = !p.h0;  // the state is zero: its products are left out

    for (int t0 = 0; t0 < len; t0 += kC) {
        const int n_tok = min(kC, len - t0);
        RowPairs<T, DK> kr, qr;
        kr.load(kp + (int64_t)t0 * p.ldk, p.ldk, n_tok, p.dk, p.vec_k);
        qr.load(qp + (int64_t)t0 * p.ldq, p.ldq, n_tok, p.dk, p.vec_k);
        T v[4][NC][4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = rt * 16 + g4 + r, c = col0 + n * 16;
                    v[rt][n][r] = t < n_tok && c < p.dv ? vp[(int64_t)(t0 + t) * p.ldv + c] : Io<T>::zero();
                }
        __syncthreads();  // the chunk before is done with LDS
        kr.store(ks, kt, rows->rk, 1.0f, p.l2norm);
        qr.store(qs, nullptr, rows->rq, p.scale, p.l2norm);
        if (wave == 0) chunk_gates<T>(gp + (int64_t)t0 * p.H, bp + (int64_t)t0 * p.H, p.H, n_tok, rows);
        __syncthreads();
        f32x4 a[3];
        chunk_products<T, DK, true>(ks, qs, rows, mt, a);
        __syncthreads();
        invert_diagonal(mt, Sh::MS, td);
        __syncthreads();
        f32x4 t[4];
        inverse_rows(mt, Sh::MS, td, t);
        store_t<T, DK, PT>(t, ts);
        // the state's products: X = K S, Y = Q S
        f32x4 X[4][NC], Y[4][NC];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n) X[rt][n] = Y[rt][n] = f32x4{0, 0, 0, 0};
        if (!zero) {
#pragma unroll
            for (int kb = 0; kb < DK / 32; ++kb) {
                Parts<T, PS> sp[NC];
#pragma unroll
                for (int n = 0; n < NC; ++n) split<PS>(S[2 * kb][n], S[2 * kb + 1][n], sp[n]);
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) {
                    const int at = (rt * 16 + l16) * Sh::KS + kb * 32 + g4 * 2;
                    const Frag<T> fk = Frag<T>::load(ks + at), fq = Frag<T>::load(qs + at);
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
#pragma unroll
                        for (int q = PS - 1; q >= 0; --q) X[rt][n] = mma(fk, sp[n].p[q], X[rt][n]);
#pragma unroll
                        for (int q = PY - 1; q >= 0; --q) Y[rt][n] = mma(fq, sp[n].p[q], Y[rt][n]);
                    }
                }
            }
        }
        // R = beta (V - e^G X), in X's place
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 be = four(rows->beta + rt * 16 + g4), eg = four(rows->eg + rt * 16 + g4),
                        rk = four(rows->rk + rt * 16 + g4);
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[rt][n][r] = be[r] * __builtin_fmaf(-(eg[r] * rk[r]), X[rt][n][r], to_f32(v[rt][n][r]));
        }
        __syncthreads();  // T is there; M is done with
        store_a<T, DK, PA>(a, as);
        f32x4 U[4][NC];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n) U[rt][n] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Parts<T, PS> rp[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) split<PS>(X[2 * kb][n], X[2 * kb + 1][n], rp[n]);
#pragma unroll
            for (int rt = 2 * kb; rt < 4; ++rt)
                mma_columns<PT, PS, NC>(ts + (rt * 16 + l16) * Sh::TS + kb * 32 + g4 * 2, kC * Sh::TS, rp, U[rt]);
        }
        __syncthreads();  // A is there
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 f = four(rows->eg + rt * 16 + g4) * four(rows->rq + rt * 16 + g4);
#pragma unroll
            for (int n = 0; n < NC; ++n) Y[rt][n] *= f;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Parts<T, PA> up[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) split<PA>(U[2 * kb][n], U[2 * kb + 1][n], up[n]);
#pragma unroll
            for (int rt = 2 * kb; rt < 4; ++rt)
                mma_columns<PA, PA, NC>(as + (rt * 16 + l16) * Sh::TS + kb * 32 + g4 * 2, kC * Sh::TS, up, Y[rt]);
        }
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t1 = rt * 16 + g4 + r, c = col0 + n * 16;
                    if (t1 < n_tok && c < p.dv) op[(int64_t)(t0 + t1) * p.H * p.dv + c] = from_f32<T>(Y[rt][n][r]);
                }
        zero = false;
        if (t0 + kC >= len && !p.hT) break;  // nobody asks for the state after the last chunk
        const float ec = rows->eg[kC - 1];
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int n = 0; n < NC; ++n) S[d][n] *= ec;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Parts<T, PS> up[NC];
#pragma unroll
            for (int n = 0; n < NC; ++n) {
                const int r0 = kb * 32 + g4;
                split<PS>(U[2 * kb][n] * (four(rows->er + r0) * four(rows->rk + r0)),
                          U[2 * kb + 1][n] * (four(rows->er + r0 + 16) * four(rows->rk + r0 + 16)), up[n]);
            }
#pragma unroll
            for (int d = 0; d < DK / 16; ++d)
                mma_columns<1, PS, NC>(kt + (d * 16 + l16) * Sh::TS + kb * 32 + g4 * 2, 0, up, S[d]);
        }
    }
    if (!p.hT) return;
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = d * 16 + g4 + r, c = col0 + n * 16;
                if (row < p.dk && c < p.dv) p.hT[sbase + (int64_t)row * p.dv + c] = S[d][n][r];
            }
}

template <typename T, int DK, int NC, int PS> hipError_t launch_delta_fwd_one(const DeltaParams& p, hipStream_t s) {
    auto kern = delta_fwd_kernel<T, DK, NC, PS>;
    constexpr int bytes = FwdLds<T, DK, PS>::bytes;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    const int tiles = (p.dv + 64 * NC - 1) / (64 * NC);
    const int64_t units = (int64_t)p.rows * p.H * tiles;
    hipLaunchKernelGGL(kern, dim3((unsigned)units), dim3(kDeltaThreads), bytes, s, p, tiles, units);
    return hipGetLastError();
}

}  // namespace sfm
