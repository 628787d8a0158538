// delta_fwd.h -- the chunked forward of the gated delta rule (kernels; one translation unit per io type).
#pragma once

#include "delta_chunk.h"

namespace sfm {

// LDS of the forward, in bytes from the start.
template <typename T, int DK, int PS> struct FwdLds {
    using Sh = ChunkShape<T, DK>;
    static constexpr int PT = PS;                                  // parts of T
    static constexpr int PA = sizeof(T) == 4 ? 1 : 2;              // parts of A
    static constexpr int frag_bytes = kLowerFrags * kFragSize * (int)sizeof(T);
    static constexpr int rows = 0;
    static constexpr int ks = (int)sizeof(ChunkRows);
    static constexpr int qs = ks + Sh::row_bytes;
    static constexpr int as = qs + Sh::row_bytes;                  // A; M before it
    static constexpr int ts = as + (PA * frag_bytes > kBytesM ? PA * frag_bytes : kBytesM);
    static constexpr int bytes = ts + PT * frag_bytes;
    static constexpr int groups = 160 * 1024 / bytes < 2 ? 1 : 2;  // workgroups to a compute unit
};

// A workgroup takes one (row, head) and 64 NC columns of its values, NC tiles of 16 to a wave, and walks the
// row's chunks; the state's columns stay in the wave's accumulators (float32) all the way.
template <typename T, int DK, int NC, int PS>
__global__ __launch_bounds__(kDeltaThreads, (FwdLds<T, DK, PS>::groups)) void delta_fwd_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    using Sh = ChunkShape<T, DK>;
    using L = FwdLds<T, DK, PS>;
    constexpr int PA = L::PA, PT = L::PT, PY = PS < 2 ? PS : 2;
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs),
      *as = reinterpret_cast<T*>(lds + L::as), *ts = reinterpret_cast<T*>(lds + L::ts);
    float* mt = reinterpret_cast<float*>(lds + L::as);

    const unsigned unit = die_local(blockIdx.x, units), rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
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
    constexpr int E = (int)sizeof(T);
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    unsigned soff[NC], voff[NC], ooff[NC];  // this lane's columns in a state, in the values and in the output
#pragma unroll
    for (int n = 0; n < NC; ++n) {
        const int c = col0 + n * 16;
        soff[n] = c < p.dv ? (unsigned)(g4 * p.dv + c) * 4u : kNowhere;
        voff[n] = c < p.dv ? (unsigned)(g4 * p.ldv + c) * E : kNowhere;
        ooff[n] = c < p.dv ? (unsigned)(g4 * p.H * p.dv + c) * E : kNowhere;
    }

    f32x4 S[DK / 16][NC];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int n = 0; n < NC; ++n) S[d][n] = f32x4{0, 0, 0, 0};
    if (p.h0) {
        const Buf b = make_buf(p.h0 + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[d][n][r] = buf_load<float>(b, fresh(soff[n]) + (unsigned)((d * 16 + r) * p.dv) * 4u);
    }
    bool zero = !p.h0;  // the state is zero: its products are left out

    for (int64_t t0 = 0; t0 < len; t0 += kC) {
        const int64_t n_tok = min((int64_t)kC, len - t0);
        RowShare<T, DK> kr, qr;
        kr.load(make_buf(kp + t0 * p.ldk, n_tok * p.ldk * E), p.ldk, p.dk, p.vec_k);
        qr.load(make_buf(qp + t0 * p.ldq, n_tok * p.ldq * E), p.ldq, p.dk, p.vec_k);
        const Buf vb = make_buf(vp + t0 * p.ldv, n_tok * p.ldv * E);
        T v[4][NC][4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[rt][n][r] = buf_load<T>(vb, fresh(voff[n]) + (unsigned)((rt * 16 + r) * p.ldv) * E);
        __syncthreads();  // the chunk before is done with LDS
        kr.store(ks, rows->rk, 1.0f, p.l2norm);
        qr.store(qs, rows->rq, p.scale, p.l2norm);
        if (wave == 0) chunk_gates<T>(gp + t0 * p.H, bp + t0 * p.H, p.H, (int)n_tok, rows);
        __syncthreads();
        f32x4 a[3];
        chunk_products<T, DK>(ks, qs, rows, mt, a);
        __syncthreads();
        invert_diagonal(mt);
        __syncthreads();
        f32x4 t[4];
        inverse_rows(mt, t);
        store_t<PT>(t, ts);
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
                    const int at = (rt * 16 + l16) * Sh::KS + kb * 32 + g4;
                    const Frag<T> fk = load_runs<T>(ks + at), fq = load_runs<T>(qs + at);
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
        store_a<PA>(a, as);
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
                mma_parts<PT, PS, NC>(load_parts<PT>(ts, lower_frag(rt, kb)), rp, U[rt]);
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
                mma_parts<PA, PA, NC>(load_parts<PA>(as, lower_frag(rt, kb)), up, Y[rt]);
        }
        const Buf ob = make_buf(op + (int64_t)t0 * p.H * p.dv, (int64_t)n_tok * p.H * p.dv * E);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int n = 0; n < NC; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_store<T>(ob, fresh(ooff[n]) + (unsigned)((rt * 16 + r) * p.H * p.dv) * E, from_f32<T>(Y[rt][n][r]));
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
                mma_parts<1, PS, NC>(Parts<T, 1>{load_transposed<T>(ks + kb * 32 * Sh::KS + d * 16, Sh::KS)}, up, S[d]);
        }
    }
    if (!p.hT) return;
    const Buf sb = make_buf(p.hT + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) buf_store<float>(sb, fresh(soff[n]) + (unsigned)((d * 16 + r) * p.dv) * 4u, S[d][n][r]);
}

template <typename T, int DK, int NC, int PS> hipError_t launch_delta_fwd_one(const DeltaParams& p, hipStream_t s) {
    auto kern = delta_fwd_kernel<T, DK, NC, PS>;
    constexpr int bytes = FwdLds<T, DK, PS>::bytes;
    if (bytes > 64 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    const unsigned tiles = (p.dv + 64 * NC - 1) / (64 * NC), units = (unsigned)p.rows * p.H * tiles;
    hipLaunchKernelGGL(kern, dim3(units), dim3(kDeltaThreads), bytes, s, p, tiles, units);
    return hipGetLastError();
}

}  // namespace sfm
