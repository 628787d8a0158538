// delta_bwd.h -- the backward of the gated delta rule by chunks (kernels; one translation unit per io type).
//
// With the forward's names (delta_chunk.h; q' = scale q, both after their norm), dO given and dS' the gradient of
// the state after the chunk:
//     dU = A^T dO + e^(G_C - G) K dS',       dR = T^T dU,        dV = beta dR,
//     dS0 = e^(G_C) dS' + Q'^T (e^G dO) - K^T (beta e^G dR),
//     dA = lower part of dO U^T,             dM = -strictly lower part of dR U^T,
//     dq' = e^G dO S0^T + (dA D) K,
//     dk  = -beta e^G dR S0^T + e^(G_C - G) U dS'^T + (dA D)^T Q' + W K + W^T K,   W_ij = beta_i D_ij dM_ij,
//     dbeta_i = dR_i.V_i - e^(G_i) k_i.(S0 dR_i) + sum_j dM_ij D_ij k_i.k_j,
//     dG_i = sum_j (P_ij - P_ji) + e^(G_i) q'_i.(S0 dO_i) - beta_i e^(G_i) k_i.(S0 dR_i) - c_i,
//         P = dA A + dM M,  c_i = e^(G_C - G_i) k_i.(dS' U_i),
//     dG_C += sum_i c_i + e^(G_C) <S0, dS'>,    dg = sums of dG from the token to the chunk's end.
// Four passes: the preparing kernel (T, A), the walk forward (states before the chunks, U), the walk back below
// (dS', dR, dV, the state's gradient) and, a workgroup to every chunk and head, the rest.  The walks are bound as the
// forward's (a chunk's latency); the last pass reads 4 bytes of every state and gradient value (260 KB to a chunk and
// head of 128 x 128) with two workgroups to a unit, 3.6 TB/s.  64 rows x 198 tokens x 5 heads of 64: 101 us = 17
// preparing + 42 walks + 42 (float32, 16 rows: 84 = 11 + 33 + 40); 2 x 4002 x 8 heads of 128 over 4 key heads: 246 us =
// 19 + 137 + 72 + 18 for the sums over shared heads.
#pragma once

#include "delta_narrow.h"

namespace sfm {

// The walk back: as the walk forward, a workgroup to a (row, head) and 64 columns, from the last chunk to the first.
template <typename T, int DK, int P>
__device__ __forceinline__ void reverse(const DeltaParams& p, unsigned tiles, unsigned unit) {
    using Sh = ChunkShape<T, DK>;
    using L = WalkLds<T, DK, P>;
    using Ops = ChunkOperands<T, P>;
    constexpr int PW = P < 2 ? P : 2;
    constexpr int E = (int)sizeof(T);
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs),
      *as = reinterpret_cast<T*>(lds + L::as), *ts = reinterpret_cast<T*>(lds + L::ts);

    const unsigned rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int col = (int)(unit - rh * tiles) * 64 + wave * 16 + l16;
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
    const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
    const int64_t obase = (first * p.H + h) * p.dv, ldo = (int64_t)p.H * p.dv;
    const T* gop = static_cast<const T*>(p.dout) + obase;
    T* dvp = static_cast<T*>(p.dv_) + obase;
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    const unsigned soff = col < p.dv ? (unsigned)(g4 * p.dv + col) * 4u : kNowhere;
    const unsigned ooff = col < p.dv ? (unsigned)(g4 * ldo + col) * E : kNowhere;
    const int64_t entry0 = (int64_t)chunk_entry(p, s, first) * p.H + h;
    const int vals = (int)tiles * 64;

    f32x4 dS[DK / 16];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) dS[d] = f32x4{0, 0, 0, 0};
    if (p.dhT) {
        const Buf b = make_buf(p.dhT + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) dS[d][r] = buf_load<float>(b, fresh(soff) + (unsigned)((d * 16 + r) * p.dv) * 4u);
    }

    RowShare<T, DK> kr, qr;
    Linear<Ops::bytes> ops;
    unsigned v[4][4];
    auto fetch = [&](int c) {
        const int64_t t0 = (int64_t)c * kC, n = min((int64_t)kC, len - t0);
        kr.load(make_buf(kp + t0 * p.ldk, n * p.ldk * E), p.ldk, p.dk, p.vec_k);
        qr.load(make_buf(qp + t0 * p.ldq, n * p.ldq * E), p.ldq, p.dk, p.vec_k);
        ops.load(p.w_ops + (entry0 + (int64_t)c * p.H) * Ops::bytes);
        const Buf ob = make_buf(gop + t0 * ldo, n * ldo * E);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[rt][r] = buf_load_bits<T>(ob, fresh(ooff) + (unsigned)((rt * 16 + r) * ldo) * E);
    };
    static_assert(L::as == Ops::a, "T and A lie in LDS as in the workspace");
    int c = (len + kC - 1) / kC - 1;
    if (c >= 0) fetch(c);

    for (; c >= 0; --c) {
        const int64_t t0 = (int64_t)c * kC, n_tok = min((int64_t)kC, len - t0), here = entry0 + (int64_t)c * p.H;
        lds_barrier();  // the chunk after is done with LDS
        kr.store(ks, nullptr, 0);
        qr.store(qs, nullptr, 0);
        ops.store(lds);
        lds_barrier();
        // dO as an operand and, by e^G q', for the state
        Parts<T, 1> go[2];
        f32x4 gov[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int r = 0; r < 4; ++r) gov[rt][r] = Io<T>::of_bits(v[rt][r]);
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) split<1>(gov[2 * kb], gov[2 * kb + 1], go[kb]);  // (exact)
        if (c > 0) fetch(c - 1);

        f32x4 dU[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) dU[rt] = f32x4{0, 0, 0, 0};
        {
            Frag<T> fk[2][4];
            auto load = [&](int kb) {
#pragma unroll
                for (int rt = 0; rt < 4; ++rt) fk[kb & 1][rt] = load_runs<T>(ks + (rt * 16 + l16) * Sh::KS + kb * 32 + g4);
            };
            load(0);
#pragma unroll
            for (int kb = 0; kb < DK / 32; ++kb) {
                if (kb + 1 < DK / 32) load(kb + 1);
                loads_end();
                Parts<T, P> sp;
                split<P>(dS[2 * kb], dS[2 * kb + 1], sp);
                store_planes<PW>(sp, reinterpret_cast<T*>(p.w_ds) + here * PW * vals * DK + (int64_t)col * DK + kb * 32 + g4, (int64_t)vals * DK);
#pragma unroll
                for (int q = P - 1; q >= 0; --q)
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) dU[rt] = mma(fk[kb & 1][rt], sp.p[q], dU[rt]);
            }
        }
        {
            Parts<T, P> at[kLowerFrags];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int kb = jt / 2; kb < 2; ++kb) at[upper_frag(jt, kb)] = load_parts_transposed<P>(as, jt, kb);
            loads_end();
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) dU[rt] *= four(rows->er + rt * 16 + g4) * four(rows->rk + rt * 16 + g4);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) mma_upper<P, 1>(at, go[kb], kb, dU);
        }
        f32x4 dR[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) dR[rt] = f32x4{0, 0, 0, 0};
        {
            Parts<T, P> tt[kLowerFrags], up[2];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt)
#pragma unroll
                for (int kb = jt / 2; kb < 2; ++kb) tt[upper_frag(jt, kb)] = load_parts_transposed<P>(ts, jt, kb);
            loads_end();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) split<P>(dU[2 * kb], dU[2 * kb + 1], up[kb]);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) mma_upper<P, P>(tt, up[kb], kb, dR);
        }
        const Buf db = make_buf(dvp + t0 * ldo, n_tok * ldo * E);
        Parts<T, P> wk[2], wq[2];
        f32x4 wkv[4], wqv[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
            const f32x4 be = four(rows->beta + rt * 16 + g4), eg = four(rows->eg + rt * 16 + g4);
            const f32x4 gv = be * dR[rt];
#pragma unroll
            for (int r = 0; r < 4; ++r) buf_store<T>(db, fresh(ooff) + (unsigned)((rt * 16 + r) * ldo) * E, from_f32<T>(gv[r]));
            wkv[rt] = gv * (-eg * four(rows->rk + rt * 16 + g4));
            wqv[rt] = gov[rt] * (eg * four(rows->rq + rt * 16 + g4) * p.scale);
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            Parts<T, PW> rp;
            split<PW>(dR[2 * kb], dR[2 * kb + 1], rp);
            store_planes<PW>(rp, reinterpret_cast<T*>(p.w_dr) + here * PW * vals * kC + (int64_t)col * kC + kb * 32 + g4, (int64_t)vals * kC);
        }
        if (c == 0 && !p.dh0) break;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            split<P>(wkv[2 * kb], wkv[2 * kb + 1], wk[kb]);
            split<P>(wqv[2 * kb], wqv[2 * kb + 1], wq[kb]);
        }
        const float ec = rows->eg[kC - 1];
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) dS[d] *= ec;
#pragma unroll
        for (int d0 = 0; d0 < DK / 16; d0 += 2) {
            Frag<T> fk[2][2], fq[2][2];
#pragma unroll
            for (int d = 0; d < 2; ++d)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    fk[d][kb] = load_transposed<T>(ks + kb * 32 * Sh::KS + (d0 + d) * 16, Sh::KS);
                    fq[d][kb] = load_transposed<T>(qs + kb * 32 * Sh::KS + (d0 + d) * 16, Sh::KS);
                }
            loads_end();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int q = P - 1; q >= 0; --q)
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        dS[d0 + d] = mma(fk[d][kb], wk[kb].p[q], dS[d0 + d]);
                        dS[d0 + d] = mma(fq[d][kb], wq[kb].p[q], dS[d0 + d]);
                    }
        }
    }
    if (!p.dh0) return;
    const Buf sb = make_buf(p.dh0 + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) buf_store<float>(sb, fresh(soff) + (unsigned)((d * 16 + r) * p.dv) * 4u, dS[d][r]);
}

// The same with few columns to a workgroup (delta_narrow.h): the waves that carry the state's gradient sum K dS' over
// their keys, and the others bring the operands and make what does not hang on the state a chunk ahead: A^T dO and
// Q^T (e^G scale dO).  T lies in LDS for its transposing reads (bfloat16) or is gathered from memory (float32).
template <typename T, int DK, int P> struct ReverseNarrowLds {
    using Sh = ChunkShape<T, DK>;
    using N = NarrowShape<DK>;
    static constexpr int E = (int)sizeof(T), frag = kFragSize * E, lower = P * kLowerFrags * frag, ex = N::CT * 2 * frag;
    static constexpr int ks = (int)sizeof(ChunkRows), ts = ks + Sh::row_bytes, half = ts + (E == 2 ? lower : 0);
    static constexpr int as = 2 * half, qs = as + lower, gs = qs + Sh::row_bytes, wq = gs + ex, up = wq + P * ex, wk = up + P * ex,
                         xp = wk + P * ex, za = xp + 16 * 1024, zq = za + N::CT * 4 * 1024, bytes = zq + 8 * 1024;
    static_assert(bytes <= 160 * 1024, "fits a compute unit");
};

// load_parts_transposed from memory, float32
__device__ __forceinline__ Frag<float> gather_transposed(const Buf& b, unsigned base, int jt, int kb) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    f32x4 x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int it = 2 * kb + i;
        const int e = lower_frag(it, jt >> 1) * kFragSize + ((l16 >> 2) * 16 + g4) * 8 + (jt & 1) * 4 + (l16 & 3);
        const unsigned at = fresh(it >= jt ? base + (unsigned)e * 4u : kNowhere);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = buf_load<float>(b, at + (unsigned)j * 32u);
    }
    return Frag<float>{x[0], x[1]};
}

template <typename T, int DK, int P, bool VEC>
__device__ __forceinline__ void narrow_reverse(const DeltaParams& p, unsigned tiles, unsigned unit) {
    constexpr int PW = P < 2 ? P : 2, E = (int)sizeof(T);
    using Sh = ChunkShape<T, DK>;
    using Ops = ChunkOperands<T, P>;
    using N = NarrowShape<DK>;
    using L = ReverseNarrowLds<T, DK, P>;
    constexpr int CT = N::CT, KW = N::KW, NF = CT * 2;
    extern __shared__ char lds[];
    const int wave = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    const N my(wave & 3);

    const unsigned rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const int chunks = (len + kC - 1) / kC;
    const int64_t entry0 = (int64_t)chunk_entry(p, s, first) * p.H + h;
    T *up = reinterpret_cast<T*>(lds + L::up), *wk = reinterpret_cast<T*>(lds + L::wk), *wq = reinterpret_cast<T*>(lds + L::wq),
      *gs = reinterpret_cast<T*>(lds + L::gs);
    f32x4 *xp = reinterpret_cast<f32x4*>(lds + L::xp) + lane, *za = reinterpret_cast<f32x4*>(lds + L::za) + lane,
          *zq = reinterpret_cast<f32x4*>(lds + L::zq) + lane;
    auto half_of = [&](int i) { return lds + (i & 1 ? L::half : 0); };
    const int col = (int)(unit - rh * tiles) * N::cols + my.cw * 16 + l16;
    const int64_t obase = (first * p.H + h) * p.dv, ldo = (int64_t)p.H * p.dv;
    // rows of the transposed triangle: the upper tiles have both steps of 32 columns, the lower ones the second
    auto both = [&](int i) { return CT == 2 ? i == 0 : my.kw < 2; };

    if (wave >= 4) {  // step i is chunk chunks - 1 - i
        if (chunks <= 0) return;
        const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
        const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
        const T* gop = static_cast<const T*>(p.dout) + obase;
        RowShare<T, DK> kr, qr;
        Linear<(int)sizeof(ChunkRows)> scalars;
        Linear<L::lower> ta, tt;
        unsigned v[CT][4];
        f32x4 eg[CT], rq[CT], Za[CT], Zq[2];
        auto load_k = [&](int i) {  // (behind the row's end the buffers are empty)
            const bool in = i < chunks;
            const int c = in ? chunks - 1 - i : 0;
            const int64_t t = (int64_t)c * kC, n = in ? min((int64_t)kC, len - t) : 0;
            const char* o = p.w_ops + (entry0 + (int64_t)c * p.H) * Ops::bytes;
            kr.load(make_buf(kp + t * p.ldk, n * p.ldk * E), p.ldk, p.dk, VEC);
            scalars.load(o, in);
            if constexpr (E == 2) tt.load(o + Ops::t, in);
        };
        auto store_k = [&](char* to) {
            kr.store(reinterpret_cast<T*>(to + L::ks), nullptr, 0);
            scalars.store(to);
            if constexpr (E == 2) tt.store(to + L::ts);
        };
        auto load_q = [&](int i) {
            const bool in = i < chunks;
            const int c = in ? chunks - 1 - i : 0;
            const int64_t t = (int64_t)c * kC, n = in ? min((int64_t)kC, len - t) : 0;
            const char* o = p.w_ops + (entry0 + (int64_t)c * p.H) * Ops::bytes;
            const Buf ob = make_buf(gop + t * ldo, n * ldo * E), rb = make_buf(o, in ? sizeof(ChunkRows) : 0);
            typedef unsigned word4 __attribute__((ext_vector_type(4)));
            qr.load(make_buf(qp + t * p.ldq, n * p.ldq * E), p.ldq, p.dk, VEC);
            ta.load(o + Ops::a, in);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int tok = my.tile(j) * 16 + g4;
                const unsigned at = fresh(col < p.dv ? (unsigned)(tok * ldo + col) * E : kNowhere);
#pragma unroll
                for (int r = 0; r < 4; ++r) v[j][r] = buf_load_bits<T>(ob, at + (unsigned)(r * ldo) * E);
                eg[j] = __builtin_bit_cast(f32x4, buf_load<word4>(rb, (unsigned)(offsetof(ChunkRows, eg) + tok * 4)));
                rq[j] = __builtin_bit_cast(f32x4, buf_load<word4>(rb, (unsigned)(offsetof(ChunkRows, rq) + tok * 4)));
            }
        };
        auto store_q = [&] {  // Q, A and dO, as it is and by e^G scale
            qr.store(reinterpret_cast<T*>(lds + L::qs), nullptr, 0);
            ta.store(lds + L::as);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int t = my.tile(j);
                f32x4 x;
#pragma unroll
                for (int r = 0; r < 4; ++r) x[r] = Io<T>::of_bits(v[j][r]);
                store_half<1, NF>(x, gs, my.cw * 2 + (t >> 1), t & 1);
                store_half<P, NF>(x * (eg[j] * rq[j] * p.scale), wq, my.cw * 2 + (t >> 1), t & 1);
            }
        };
        auto products = [&] {
            const T *as = reinterpret_cast<const T*>(lds + L::as), *qs = reinterpret_cast<const T*>(lds + L::qs) + my.kw * 32;
            Parts<T, 1> go[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) go[kb] = load_exchange<1, NF>(gs, my.cw * 2 + kb);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 x[3];
                zero3(x);
                if (both(j)) mma_spread<P, 1>(load_parts_transposed<P>(as, my.tile(j), 0), go[0], x, 0);
                mma_spread<P, 1>(load_parts_transposed<P>(as, my.tile(j), 1), go[1], x, 0);
                Za[j] = gather3(x);
            }
            Parts<T, P> fv[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) fv[kb] = load_exchange<P, NF>(wq, my.cw * 2 + kb);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                f32x4 x[3];
                zero3(x);
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) {
                    const Parts<T, 1> tq = {{load_eight_transposed<T>(qs + kb * 32 * Sh::KS, Sh::KS, d)}};
                    mma_spread<1, P>(tq, fv[kb], x, 0);
                }
                Zq[d] = gather3(x);
            }
        };
        auto store_za = [&] {
#pragma unroll
            for (int j = 0; j < CT; ++j) za[(my.cw * 4 + my.tile(j)) * 64] = Za[j];
        };
        load_q(0);
        load_k(0);
        store_q();
        store_k(lds);
        load_q(1);
        load_k(1);
        lds_barrier();
        products();
        store_za();
        for (int i = 0; i < chunks; ++i) {
            lds_barrier();
#pragma unroll
            for (int d = 0; d < 2; ++d) zq[((wave & 3) * 2 + d) * 64] = Zq[d];
            store_q();
            load_q(i + 2);
            lds_barrier();
            products();
            store_k(half_of(i + 1));
            lds_barrier();
            store_za();
            load_k(i + 2);
        }
        return;
    }

    T* dvp = static_cast<T*>(p.dv_) + obase;
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    const int key = my.kw * 32 + 2 * g4;
    const unsigned soff = col < p.dv ? (unsigned)(key * p.dv + col) * 4u : kNowhere;
    const int vals = (p.dv + 63) / 64 * 64;

    f32x4 dS[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) dS[d] = f32x4{0, 0, 0, 0};
    if (p.dhT) {
        const Buf b = make_buf(p.dhT + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) dS[d][r] = buf_load<float>(b, soff + (unsigned)((d * 4 + r) * p.dv) * 4u);
    }
    Parts<T, 1> fk[4];  // K's rows, this wave's keys, of the chunk to come
    auto load_k = [&](int i) {
        const T* ks = reinterpret_cast<const T*>(half_of(i) + L::ks) + my.kw * 32 + l16 * Sh::KS + 2 * g4;
#pragma unroll
        for (int t = 0; t < 4; ++t) fk[t].p[0] = load_eight<T>(ks + t * 16 * Sh::KS);
    };
    if (chunks > 0) {
        lds_barrier();
        load_k(0);
    }

    for (int i = 0; i < chunks; ++i) {
        const int c = chunks - 1 - i;
        const int64_t t0 = (int64_t)c * kC, n_tok = min((int64_t)kC, len - t0), entry = entry0 + (int64_t)c * p.H;
        const char* half = half_of(i);
        const ChunkRows* rows = reinterpret_cast<const ChunkRows*>(half);
        const T* ks = reinterpret_cast<const T*>(half + L::ks);
        // K dS' over this wave's keys
        {
            Parts<T, P> fs;
            split<P>(dS[0], dS[1], fs);
            f32x4 x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
                for (int t = 0; t < 4; ++t) x[t] = mma(fk[t].p[0], fs.p[q], x[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t) xp[((my.cw * 4 + t) * KW + my.kw) * 64] = x[t];
            store_eight<PW>(fs, reinterpret_cast<T*>(p.w_ds) + entry * PW * vals * DK + (int64_t)col * DK + key, (int64_t)vals * DK);
        }
        f32x4 er[CT], be[CT], fw[CT];
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int tok = my.tile(j) * 16 + g4;
            er[j] = four(rows->er + tok) * four(rows->rk + tok);
        }
        lds_barrier();
        // dU = e^(G_C - G) K dS' + A^T dO
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int t = my.tile(j);
            f32x4 x[KW];
#pragma unroll
            for (int k = 0; k < KW; ++k) x[k] = xp[((my.cw * 4 + t) * KW + k) * 64];
            const f32x4 z = za[(my.cw * 4 + t) * 64];
            f32x4 sum = x[0] + x[1];
            if constexpr (KW == 4) sum += x[2] + x[3];
            store_half<P, NF>(sum * er[j] + z, up, my.cw * 2 + (t >> 1), t & 1);
        }
        Parts<T, P> tt[CT][2];
        if constexpr (E == 2) {
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (CT == 1 || kb == 1 || j == 0)
                        tt[j][kb] = load_parts_transposed<P>(reinterpret_cast<const T*>(half + L::ts), my.tile(j), both(j) ? kb : 1);
        } else {
            const Buf tb = make_buf(p.w_ops + entry * Ops::bytes, Ops::bytes);
#pragma unroll
            for (int j = 0; j < CT; ++j)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (CT == 1 || kb == 1 || j == 0) tt[j][kb].p[0] = gather_transposed(tb, Ops::t, my.tile(j), both(j) ? kb : 1);
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int tok = my.tile(j) * 16 + g4;
            be[j] = four(rows->beta + tok);
            fw[j] = -four(rows->eg + tok) * four(rows->rk + tok);
        }
        lds_barrier();
        // dR = T^T dU
        f32x4 dR[CT];
        {
            Parts<T, P> fu[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) fu[kb] = load_exchange<P, NF>(up, my.cw * 2 + kb);
            loads_end();
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                f32x4 x[3];
                zero3(x);
                if (both(j)) mma_spread<P, P>(tt[j][0], fu[0], x, 0);
                mma_spread<P, P>(tt[j][1], fu[1], x, 0);
                dR[j] = gather3(x);
            }
        }
        Parts<T, 1> kt[2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int d = 0; d < 2; ++d) kt[d][kb].p[0] = load_eight_transposed<T>(ks + kb * 32 * Sh::KS + my.kw * 32, Sh::KS, d);
        loads_end();
        const Buf db = make_buf(dvp + t0 * ldo, n_tok * ldo * E);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int t = my.tile(j);
            const f32x4 gv = be[j] * dR[j];
            store_half<P, NF>(gv * fw[j], wk, my.cw * 2 + (t >> 1), t & 1);
            const unsigned at = fresh(col < p.dv ? (unsigned)((t * 16 + g4) * ldo + col) * E : kNowhere);
#pragma unroll
            for (int r = 0; r < 4; ++r) buf_store<T>(db, at + (unsigned)(r * ldo) * E, from_f32<T>(gv[r]));
            store_four<PW>(dR[j], reinterpret_cast<T*>(p.w_dr) + entry * PW * vals * kC + (int64_t)col * kC + t * 16 + g4, (int64_t)vals * kC);
        }
        const float ec = rows->eg[kC - 1];
        lds_barrier();
        // dS = e^(G_C) dS' + K^T (-beta e^G dR) + Q^T (e^G scale dO)
        Parts<T, P> fv[2];
        f32x4 z[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) fv[kb] = load_exchange<P, NF>(wk, my.cw * 2 + kb);
#pragma unroll
        for (int d = 0; d < 2; ++d) z[d] = zq[(wave * 2 + d) * 64];
        if (CT == 1) load_k(i + 1);
        loads_end();
        if (c > 0 || p.dh0) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                f32x4 x[3];
                zero3(x);
                x[0] = dS[d] * ec + z[d];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) mma_spread<1, P>(kt[d][kb], fv[kb], x, 0);
                dS[d] = gather3(x);
            }
        }
        if (CT > 1) {
            loads_end();
            load_k(i + 1);
        }
    }
    if (!p.dh0) return;
    const Buf sb = make_buf(p.dh0 + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) buf_store<float>(sb, soff + (unsigned)((d * 4 + r) * p.dv) * 4u, dS[d][r]);
}

// Both walks in one launch: they need nothing of each other, and each alone often leaves units idle (2 x 4002 tokens,
// 8 heads of 128: 88 us and 125 us one after the other, 137 us together).
template <typename T, int DK, int P>
__global__ __launch_bounds__(kDeltaThreads, (DK == 64 ? WalkLds<T, DK, P>::groups : 1)) void delta_walks_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    if (blockIdx.x < units)  // (the longer one first)
        reverse<T, DK, P>(p, tiles, row_unit(p, blockIdx.x, units, tiles * p.H, tiles * p.share));
    else
        walk<T, DK, P, kStates>(p, tiles, row_unit(p, blockIdx.x - units, units, tiles * p.H, tiles * p.share));
}
template <typename T, int DK, int P, bool VEC>
__global__ __launch_bounds__(kNarrowThreads, 2) void delta_narrow_walks_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    if (blockIdx.x < units)
        narrow_reverse<T, DK, P, VEC>(p, tiles, row_unit(p, blockIdx.x, units, tiles * p.H, tiles * p.share));
    else
        narrow_walk<T, DK, P, kStates, VEC>(p, tiles, row_unit(p, blockIdx.x - units, units, tiles * p.H, tiles * p.share));
}

// ---------------------------------------------------------------- per chunk and head
constexpr int kVals = 32;  // values to a step of the first phase

template <typename T, int DK, int PW> struct GradLds {
    using Sh = ChunkShape<T, DK>;
    static constexpr int E = (int)sizeof(T);
    static constexpr int VS = ChunkShape<T, kVals>::KS;    // pitch of [token][value]
    static constexpr int TS = kC + 16 / E;                 // pitch of [value][token]
    static constexpr int rows = 0;
    static constexpr int sums = (int)sizeof(ChunkRows);    // float arrays [64]: see Sums
    static constexpr int work = sums + 11 * kC * 4;
    // first phase
    static constexpr int go = work, v = go + kC * VS * E, u = v + kC * VS * E, dr = u + PW * kVals * TS * E,
                         s0 = dr + PW * kVals * TS * E, ds = s0 + PW * kVals * Sh::KS * E, end1 = ds + PW * kVals * Sh::KS * E;
    // second phase
    static constexpr int ks = work, qs = ks + Sh::row_bytes, x = qs + Sh::row_bytes,
                         w = x + PW * kLowerFrags * kFragSize * E, end2 = w + PW * kLowerFrags * kFragSize * E;
    static constexpr int bytes = end1 > end2 ? end1 : end2;
};

// Planes [PW][kVals rows][LEN] of the workspace, `plane` elements apart: through registers into LDS of pitch PITCH.
template <typename T, int PW, int LEN, int PITCH> struct PlaneBlock {
    static constexpr int per = 16 / (int)sizeof(T), kRow = LEN / per, kUnits = kVals * kRow / kDeltaThreads;
    static_assert(kUnits * kDeltaThreads == kVals * kRow, "whole units to a thread");
    typedef T piece __attribute__((ext_vector_type(per)));
    piece x[PW][kUnits];
    __device__ __forceinline__ void load(const T* p, int64_t plane) {
#pragma unroll
        for (int q = 0; q < PW; ++q)
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
                x[q][i] = *reinterpret_cast<const piece*>(p + q * plane + (threadIdx.x + i * kDeltaThreads) * per);
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int q = 0; q < PW; ++q)
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                const int u = threadIdx.x + i * kDeltaThreads;
                *reinterpret_cast<piece*>(p + (q * kVals + u / kRow) * PITCH + u % kRow * per) = x[q][i];
            }
    }
    __device__ __forceinline__ float value(int i, int e) const {
        float v = 0.0f;
#pragma unroll
        for (int q = PW - 1; q >= 0; --q) v += to_f32((T)x[q][i][e]);
        return v;
    }
};

// parts of rows 16 tile .. + 15 of a [value][row] block, contraction over its 32 values
template <int PW, typename T> __device__ __forceinline__ Parts<T, PW> load_block(const T* p, int tile, int pitch) {
    Parts<T, PW> a;
#pragma unroll
    for (int q = 0; q < PW; ++q) a.p[q] = load_transposed<T>(p + q * kVals * pitch + tile * 16, pitch);
    return a;
}

// c[n] += a b[n], the products of parts as in mma_lower
template <int PA, int PB, int N, typename T>
__device__ __forceinline__ void mma_all(const Parts<T, PA>& a, const Parts<T, PB> (&b)[N], f32x4* c) {
    constexpr int top = PA > PB ? PA : PB;
#pragma unroll
    for (int p = PA - 1; p >= 0; --p)
#pragma unroll
        for (int q = PB - 1; q >= 0; --q)
            if (p + q < top)
#pragma unroll
                for (int n = 0; n < N; ++n) c[n] = mma(a.p[p], b[n].p[q], c[n]);
}

// A workgroup to every chunk and head, sixteen tokens to a wave.  First phase: the products over values (with S0,
// dS', U, dR of the workspace), 32 values at a time; second: those over tokens (with K and Q).
template <typename T, int DK, int PW>
__global__ __launch_bounds__(kDeltaThreads, (sizeof(T) == 2 ? 2 : 1)) void delta_grads_kernel(const DeltaParams p, unsigned entries, unsigned units, int ops_bytes) {
    using Sh = ChunkShape<T, DK>;
    using L = GradLds<T, DK, PW>;
    constexpr int E = (int)sizeof(T), ND = DK / 16;
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    float* sums = reinterpret_cast<float*>(lds + L::sums);
    // by token: P's row sums, the other terms of dG, c, dbeta's two halves, dR.V; P's column sums by wave; <S0, dS'>
    float *row_p = sums, *row_o = sums + kC, *row_c = sums + 2 * kC, *row_b = sums + 3 * kC, *row_e = sums + 4 * kC,
          *row_v = sums + 5 * kC, *col_p = sums + 6 * kC, *frob = sums + 10 * kC;
    const unsigned unit = row_unit(p, blockIdx.x, units, entries / (unsigned)p.rows * p.H, p.share);
    const int h = (int)(unit % (unsigned)p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    ChunkAt at;
    if (!chunk_at(p, unit / (unsigned)p.H, at)) return;
    const int64_t n = min((int64_t)kC, at.len - at.t0), tok = at.first + at.t0, entry = unit;  // (entry and head)
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int vals = (p.dv + 63) / 64 * 64;

    {
        Linear<(int)sizeof(ChunkRows)> r;
        r.load(p.w_ops + entry * ops_bytes);
        r.store(lds);
    }
    col_p[threadIdx.x] = 0.0f;

    f32x4 dq[ND], dkr[ND], dku[ND], da[4], dm[4], rv = {0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < ND; ++d) dq[d] = dkr[d] = dku[d] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) da[j] = dm[j] = f32x4{0, 0, 0, 0};
    float fr = 0.0f;
    {
        T *gs = reinterpret_cast<T*>(lds + L::go), *vs = reinterpret_cast<T*>(lds + L::v), *us = reinterpret_cast<T*>(lds + L::u),
          *rs = reinterpret_cast<T*>(lds + L::dr), *s0 = reinterpret_cast<T*>(lds + L::s0), *ds = reinterpret_cast<T*>(lds + L::ds);
        const T* ws = reinterpret_cast<const T*>(p.w_s) + entry * PW * vals * DK;
        const T* wd = reinterpret_cast<const T*>(p.w_ds) + entry * PW * vals * DK;
        const T* wu = reinterpret_cast<const T*>(p.w_u) + entry * PW * vals * kC;
        const T* wr = reinterpret_cast<const T*>(p.w_dr) + entry * PW * vals * kC;
        const T* gop = static_cast<const T*>(p.dout) + (tok * p.H + h) * p.dv;
        const T* vp = static_cast<const T*>(p.v) + tok * p.ldv + (int64_t)h * p.dv;
        RowShare<T, kVals> gr, vr;
        PlaneBlock<T, PW, DK, Sh::KS> bs, bd;
        PlaneBlock<T, PW, kC, L::TS> bu, br;
        auto fetch = [&](int v0) {
            gr.load(make_buf(gop + v0, n * p.H * p.dv * E - v0 * E), (int64_t)p.H * p.dv, p.dv - v0, p.vec_o);
            vr.load(make_buf(vp + v0, n * p.ldv * E - v0 * E), p.ldv, p.dv - v0, p.vec_v);
            bs.load(ws + (int64_t)v0 * DK, (int64_t)vals * DK);
            bd.load(wd + (int64_t)v0 * DK, (int64_t)vals * DK);
            bu.load(wu + (int64_t)v0 * kC, (int64_t)vals * kC);
            br.load(wr + (int64_t)v0 * kC, (int64_t)vals * kC);
        };
        constexpr bool ahead = DK == 64 || sizeof(T) == 4;  // (else the registers are another workgroup's)
        if (ahead) fetch(0);
        for (int v0 = 0; v0 < p.dv; v0 += kVals) {
            if (!ahead) fetch(v0);
            lds_barrier();
            gr.store(gs, nullptr, 0);
            vr.store(vs, nullptr, 0);
            bs.store(s0);
            bd.store(ds);
            bu.store(us);
            br.store(rs);
#pragma unroll
            for (int i = 0; i < bs.kUnits; ++i)
#pragma unroll
                for (int e = 0; e < bs.per; ++e) fr = __builtin_fmaf(bs.value(i, e), bd.value(i, e), fr);
            lds_barrier();
            if (ahead && v0 + kVals < p.dv) fetch(v0 + kVals);
            const Parts<T, 1> fg[1] = {{load_runs<T>(gs + (wave * 16 + l16) * L::VS + g4)}};
            const Parts<T, 1> fv[1] = {{load_runs<T>(vs + (wave * 16 + l16) * L::VS + g4)}};
            const Parts<T, PW> fr_[1] = {load_block<PW>(rs, wave, L::TS)}, fu = load_block<PW>(us, wave, L::TS);
            loads_end();
            mma_all<PW, 1>(fr_[0], fv, &rv);
#pragma unroll
            for (int d0 = 0; d0 < ND; d0 += 2) {
                Parts<T, PW> fs[2], fd[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    fs[d] = load_block<PW>(s0, d0 + d, Sh::KS);
                    fd[d] = load_block<PW>(ds, d0 + d, Sh::KS);
                }
                loads_end();
                mma_all<1, PW>(fg[0], fs, dq + d0);
                mma_all<PW, PW>(fr_[0], fs, dkr + d0);
                mma_all<PW, PW>(fu, fd, dku + d0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= wave) {
                    const Parts<T, PW> uj = load_block<PW>(us, j, L::TS);
                    mma_all<PW, 1>(uj, fg, da + j);
                    mma_all<PW, PW>(uj, fr_, dm + j);
                }
        }
    }
    // <S0, dS'> of this wave, and dR.V: the diagonal of the product
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) fr += __shfl_xor(fr, m);
    if (lane == 0) frob[wave] = fr;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (g4 + r == l16) row_v[wave * 16 + l16] = rv[r];

    // (not before: with its registers another workgroup fits on the unit)
    RowShare<T, DK> kr, qr;
    kr.load(make_buf(static_cast<const T*>(p.k) + tok * p.ldk + (int64_t)hk * p.dk, n * p.ldk * E), p.ldk, p.dk, p.vec_k);
    qr.load(make_buf(static_cast<const T*>(p.q) + tok * p.ldq + (int64_t)hk * p.dk, n * p.ldq * E), p.ldq, p.dk, p.vec_k);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs), *xs = reinterpret_cast<T*>(lds + L::x),
      *wsm = reinterpret_cast<T*>(lds + L::w);
    lds_barrier();  // the first phase's arrays are done with
    kr.store(ks, nullptr, 0);
    qr.store(qs, nullptr, 0);
    lds_barrier();

    // rows 16 wave + g4 .. + 3: the state's shares of dq', dk, dG and dbeta
    const int i0 = wave * 16 + g4;
    const f32x4 eg = four(rows->eg + i0), er = four(rows->er + i0), be = four(rows->beta + i0), rk = four(rows->rk + i0),
                rq = four(rows->rq + i0);
    {
        f32x4 sa = {0, 0, 0, 0}, se = sa, sk = sa;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float kv = to_f32(ks[(i0 + r) * Sh::KS + d * 16 + l16]), qv = to_f32(qs[(i0 + r) * Sh::KS + d * 16 + l16]);
                dq[d][r] *= eg[r];
                dkr[d][r] *= eg[r];
                dku[d][r] *= er[r];
                sa[r] = __builtin_fmaf(qv, dq[d][r], sa[r]);
                se[r] = __builtin_fmaf(kv, dkr[d][r], se[r]);
                sk[r] = __builtin_fmaf(kv, dku[d][r], sk[r]);
                dku[d][r] = __builtin_fmaf(-be[r], dkr[d][r], dku[d][r]);
            }
        f32x4 o, e, cc;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            e[r] = lanes_sum<16>(se[r]) * rk[r];
            cc[r] = lanes_sum<16>(sk[r]) * rk[r];
            o[r] = lanes_sum<16>(sa[r]) * (rq[r] * p.scale) - be[r] * e[r] - cc[r];
        }
        if (l16 == 0) {
            *reinterpret_cast<f32x4*>(row_o + i0) = o;
            *reinterpret_cast<f32x4*>(row_e + i0) = e;
            *reinterpret_cast<f32x4*>(row_c + i0) = cc;
        }
    }
    f32x4(&dk)[ND] = dku;

    // the chunk's own products, tile by tile: column i = 16 wave + l16 of the lane, rows j = 16 tj + g4 .. + 3
    f32x4 xl[4], wl[4];
    {
        const int i = wave * 16 + l16;
        const float hi = rows->ghi[i], lo = rows->glo[i], qi = rows->rq[i] * p.scale, ki = rows->rk[i], bi = rows->beta[i];
        float sp = 0.0f, sb = 0.0f;
#pragma unroll
        for (int tj = 0; tj < 4; ++tj) {
            xl[tj] = wl[tj] = f32x4{0, 0, 0, 0};
            if (tj > wave) continue;
            const f32x4 qk = rows_product<T, DK>(ks, tj, qs, wave), kk = rows_product<T, DK>(ks, tj, ks, wave);
            const int j0 = tj * 16 + g4;
            const f32x4 hj = four(rows->ghi + j0), lj = four(rows->glo + j0), kj = four(rows->rk + j0);
            f32x4 pc, xi, wi;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float d = exp2_fast((hi - hj[r]) + (lo - lj[r]));
                const float x = j0 + r <= i ? da[tj][r] * d : 0.0f;
                const float y = j0 + r < i ? -dm[tj][r] * d : 0.0f;
                const float yk = y * (ki * kj[r] * kk[r]);
                pc[r] = __builtin_fmaf(x, qi * kj[r] * qk[r], bi * yk);
                sp += pc[r];
                sb += yk;
                xl[tj][r] = x * kj[r];
                wl[tj][r] = y * (bi * kj[r]);
                xi[r] = x * qi;
                wi[r] = y * (bi * ki);
            }
            store_tile<PW>(xi, xs, wave, tj);
            store_tile<PW>(wi, wsm, wave, tj);
#pragma unroll
            for (int r = 0; r < 4; ++r) pc[r] = lanes_sum<16>(pc[r]);
            if (l16 == 0) *reinterpret_cast<f32x4*>(col_p + wave * kC + j0) = pc;
        }
        sp += __shfl_xor(sp, 16);
        sb += __shfl_xor(sb, 16);
        sp += __shfl_xor(sp, 32);
        sb += __shfl_xor(sb, 32);
        if (lane < 16) {
            row_p[i] = sp;
            row_b[i] = sb;
        }
    }
    lds_barrier();
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
        const bool low = kb <= wave / 2, up = kb >= wave / 2;
        Parts<T, PW> xp, wp, xt, wt;
        split<PW>(xl[2 * kb], xl[2 * kb + 1], xp);
        split<PW>(wl[2 * kb], wl[2 * kb + 1], wp);
        if (up) {
            xt = load_parts_transposed<PW>(xs, wave, kb);
            wt = load_parts_transposed<PW>(wsm, wave, kb);
        }
#pragma unroll
        for (int d0 = 0; d0 < ND; d0 += 2) {
            Parts<T, 1> fk[2], fq[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                fk[d].p[0] = load_transposed<T>(ks + kb * 32 * Sh::KS + (d0 + d) * 16, Sh::KS);
                fq[d].p[0] = load_transposed<T>(qs + kb * 32 * Sh::KS + (d0 + d) * 16, Sh::KS);
            }
            loads_end();
            if (low) {
                mma_all<PW, 1>(xp, fk, dq + d0);
                mma_all<PW, 1>(wp, fk, dk + d0);
            }
            if (up) {
                mma_all<PW, 1>(xt, fq, dk + d0);
                mma_all<PW, 1>(wt, fk, dk + d0);
            }
        }
    }
    // Through the norms, and out: the unit vector's gradient less its part along the vector.  A head of one key is
    // all along; what is left of it, eps / (x^2 + eps), is taken as such (the difference would have no digits).
    f32x4 tq = {0, 0, 0, 0}, tk = tq, fq = rq * p.scale, fk = rk;
    if (p.l2norm && p.dk == 1) {
        fq *= rq * rq * kDeltaNormEps;
        fk *= rk * rk * kDeltaNormEps;
    } else if (p.l2norm) {
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                tq[r] = __builtin_fmaf(to_f32(qs[(i0 + r) * Sh::KS + d * 16 + l16]), dq[d][r], tq[r]);
                tk[r] = __builtin_fmaf(to_f32(ks[(i0 + r) * Sh::KS + d * 16 + l16]), dk[d][r], tk[r]);
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            tq[r] = lanes_sum<16>(tq[r]) * (rq[r] * rq[r]);
            tk[r] = lanes_sum<16>(tk[r]) * (rk[r] * rk[r]);
        }
    }
    const bool shared = p.share > 1;
    const int heads = shared ? p.H : p.Hk, head = shared ? h : hk, size = shared ? 4 : E;
    const int64_t ld = (int64_t)heads * p.dk, base = tok * ld + (int64_t)head * p.dk;
    const Buf bq = shared ? make_buf(p.w_dq + base, n * ld * 4) : make_buf(static_cast<T*>(p.dq) + base, n * ld * E);
    const Buf bk = shared ? make_buf(p.w_dk + base, n * ld * 4) : make_buf(static_cast<T*>(p.dk_) + base, n * ld * E);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const int c = d * 16 + l16;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const unsigned at = c < p.dk ? (unsigned)((i0 + r) * ld + c) * (unsigned)size : kNowhere;
            const float kv = to_f32(ks[(i0 + r) * Sh::KS + c]), qv = to_f32(qs[(i0 + r) * Sh::KS + c]);
            const float gq = fq[r] * __builtin_fmaf(-qv, tq[r], dq[d][r]);
            const float gk = fk[r] * __builtin_fmaf(-kv, tk[r], dk[d][r]);
            if (shared) {
                buf_store<float>(bq, at, gq);
                buf_store<float>(bk, at, gk);
            } else {
                buf_store<T>(bq, at, from_f32<T>(gq));
                buf_store<T>(bk, at, from_f32<T>(gk));
            }
        }
    }
    if (wave != 0) return;
    // dg: a lane to a token, sums from the chunk's end.  (P's sums first: a row of one token that begins without a state
    // has nothing else, and its gradient is zero to the last bit.)
    float x = row_p[lane] - ((col_p[lane] + col_p[kC + lane]) + (col_p[2 * kC + lane] + col_p[3 * kC + lane])) + row_o[lane];
    float all = row_c[lane];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m);
    all += rows->eg[kC - 1] * ((frob[0] + frob[1]) + (frob[2] + frob[3]));
    if (lane == 63) x += all;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const float o = __shfl_down(x, m);
        if (lane + m < 64) x += o;
    }
    if (lane < n) {
        const int64_t at = (tok + lane) * p.H + h;
        static_cast<T*>(p.dg)[at] = from_f32<T>(x);
        static_cast<T*>(p.dbeta)[at] = from_f32<T>(row_v[lane] - row_e[lane] + row_b[lane]);
    }
}

// Shared key heads: the value heads' shares, in order.  A workgroup to every 16 tokens of a row's 64 and key head; a
// thread takes V neighbouring keys.
template <typename T, int V>
__global__ __launch_bounds__(kDeltaThreads) void delta_share_kernel(const DeltaParams p) {
    typedef float vec __attribute__((ext_vector_type(V)));
    const unsigned sq = blockIdx.x / (unsigned)p.Hk;
    const int hk = (int)(blockIdx.x - sq * (unsigned)p.Hk);
    ChunkAt at;
    if (!chunk_at(p, sq / 4, at)) return;
    const int64_t t0 = at.t0 + (sq & 3) * 16;
    const int n = (int)min((int64_t)16, at.len - t0), ct = (threadIdx.x & 31) * V;
    for (int t = threadIdx.x >> 5; t < n; t += kDeltaThreads / 32) {
        const int64_t tok = at.first + t0 + t, from = (tok * p.H + (int64_t)hk * p.share) * p.dk, to = (tok * p.Hk + hk) * p.dk;
        for (int c = ct; c < p.dk; c += 32 * V) {
            vec a, b;
#pragma unroll
            for (int e = 0; e < V; ++e) a[e] = b[e] = 0.0f;
            for (int j = 0; j < p.share; ++j) {
                a += *reinterpret_cast<const vec*>(p.w_dq + from + j * p.dk + c);
                b += *reinterpret_cast<const vec*>(p.w_dk + from + j * p.dk + c);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                static_cast<T*>(p.dq)[to + c + e] = from_f32<T>(a[e]);
                static_cast<T*>(p.dk_)[to + c + e] = from_f32<T>(b[e]);
            }
        }
    }
}

template <typename T, int DK, int P> hipError_t launch_backward(const DeltaParams& p, hipStream_t s) {
    constexpr int PW = P < 2 ? P : 2;
    hipError_t e = launch_prepare<T, DK, P, P>(p, s);
    if (e != hipSuccess) return e;
    constexpr int gb = GradLds<T, DK, PW>::bytes;
    // (few columns: those that the last pass reads, kVals at a time)
    const unsigned tiles = p.narrow ? (p.dv + kVals - 1) / kVals * (kVals / NarrowShape<DK>::cols) : (p.dv + 63) / 64;
    const unsigned units = (unsigned)p.rows * p.H * tiles;
    auto walks = !p.narrow ? delta_walks_kernel<T, DK, P>
                 : p.vec_k ? delta_narrow_walks_kernel<T, DK, P, true>
                           : delta_narrow_walks_kernel<T, DK, P, false>;
    constexpr int nb = ReverseNarrowLds<T, DK, P>::bytes, ns = WalkNarrowLds<T, DK, P, 0>::bytes;
    const int wb = p.narrow ? (nb > ns ? nb : ns) : WalkLds<T, DK, P>::bytes;
    if ((e = allow_lds(walks, wb)) != hipSuccess) return e;
    hipLaunchKernelGGL(walks, dim3(2 * units), dim3(p.narrow ? kNarrowThreads : kDeltaThreads), wb, s, p, tiles, units);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const unsigned entries = launch_entries(p), cu = entries * p.H;
    auto grads = delta_grads_kernel<T, DK, PW>;
    if ((e = allow_lds(grads, gb)) != hipSuccess) return e;
    hipLaunchKernelGGL(grads, dim3(cu), dim3(kDeltaThreads), gb, s, p, entries, cu, ChunkOperands<T, P>::bytes);
    if ((e = hipGetLastError()) != hipSuccess || p.share == 1) return e;
    const dim3 sg(entries * 4 * p.Hk);
    if (p.dk % 4 == 0)
        hipLaunchKernelGGL((delta_share_kernel<T, 4>), sg, dim3(kDeltaThreads), 0, s, p);
    else
        hipLaunchKernelGGL((delta_share_kernel<T, 1>), sg, dim3(kDeltaThreads), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
