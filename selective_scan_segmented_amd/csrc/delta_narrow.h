// delta_narrow.h -- the walks of delta_fwd.h and delta_bwd.h for few long rows: sixteen columns to a workgroup.
//
// A row's chunks follow one another, so where there are few (row, head, 64 column) workgroups the time is that of
// one chunk in one of them.  Here the four waves share sixteen columns instead of having sixteen each: wave w holds
// a quarter of the state's keys and computes the tokens 16 w .. + 15 of every product, and what the others need of it
// (the state's parts, R, U) goes through LDS in operand order.  Three barriers a chunk.  Four more waves do nothing
// but bring the next chunk's operands into the other half of LDS (where two halves fit): a compute unit moves 64
// bytes a cycle, 1000 cycles for a chunk of 66 KB, and a wave that issues such loads stands still meanwhile.
#pragma once

#include "delta_fwd.h"

namespace sfm {

// four values of a lane as half a fragment in P planes of NF fragments (half 0: slots 0..3, half 1: 4..7)
template <int P, int NF, typename T> __device__ __forceinline__ void store_half(f32x4 x, T* base, int frag, int half) {
    T* p = base + frag * kFragSize + (threadIdx.x & 63) * 8 + half * 4;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(p) = x;
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            bf16x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = (__bf16)x[j];
                x[j] -= (float)v[j];
            }
            *reinterpret_cast<bf16x4*>(p + q * NF * kFragSize) = v;
        }
    }
}
// likewise to memory: PW planes `plane` apart, and LDS, from one splitting
template <int PW, int P, int NF, typename T>
__device__ __forceinline__ void store_half_both(f32x4 x, T* base, int frag, int half, T* mem, int64_t plane) {
    T* p = base + frag * kFragSize + (threadIdx.x & 63) * 8 + half * 4;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(p) = x;
        *reinterpret_cast<f32x4*>(mem) = x;
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            bf16x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = (__bf16)x[j];
                x[j] -= (float)v[j];
            }
            *reinterpret_cast<bf16x4*>(p + q * NF * kFragSize) = v;
            if (q < PW) *reinterpret_cast<bf16x4*>(mem + q * plane) = v;
        }
    }
}
// four values of a lane as PW planes of memory
template <int PW, typename T> __device__ __forceinline__ void store_four(f32x4 x, T* mem, int64_t plane) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(mem) = x;
    } else {
#pragma unroll
        for (int q = 0; q < PW; ++q) {
            bf16x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = (__bf16)x[j];
                x[j] -= (float)v[j];
            }
            *reinterpret_cast<bf16x4*>(mem + q * plane) = v;
        }
    }
}
template <int P, int NF, typename T> __device__ __forceinline__ Parts<T, P> load_exchange(const T* base, int frag) {
    Parts<T, P> a;
#pragma unroll
    for (int q = 0; q < P; ++q) a.p[q] = Frag<T>::load(base + (q * NF + frag) * kFragSize + (threadIdx.x & 63) * 8);
    return a;
}
// c[i] += the products of parts of a and b, spread over three accumulators so that none waits for itself
template <int PA, int PB, typename T>
__device__ __forceinline__ void mma_spread(const Parts<T, PA>& a, const Parts<T, PB>& b, f32x4 (&c)[3], int from) {
    constexpr int top = PA > PB ? PA : PB;
    int i = from;
#pragma unroll
    for (int p = PA - 1; p >= 0; --p)
#pragma unroll
        for (int q = PB - 1; q >= 0; --q)
            if (p + q < top) {
                c[i % 3] = mma(a.p[p], b.p[q], c[i % 3]);
                ++i;
            }
}
__device__ __forceinline__ f32x4 gather3(const f32x4 (&c)[3]) { return (c[0] + c[1]) + c[2]; }
__device__ __forceinline__ void zero3(f32x4 (&c)[3]) { c[0] = c[1] = c[2] = f32x4{0, 0, 0, 0}; }

// LDS: NB halves of a chunk's operands, then the exchange.  PA: parts of A kept; PX: planes of the exchange's arrays
// over tokens, all together.
template <typename T, int DK, int P, int PA, int PX> struct NarrowLds {
    using Sh = ChunkShape<T, DK>;
    static constexpr int E = (int)sizeof(T);
    static constexpr int frag_bytes = kLowerFrags * kFragSize * E;
    static constexpr int ts = (int)sizeof(ChunkRows), as = ts + P * frag_bytes, ks = as + PA * frag_bytes,
                         qs = ks + Sh::row_bytes, half = qs + Sh::row_bytes;
    static constexpr int state = P * (DK / 32) * kFragSize * E, tokens = PX * 2 * kFragSize * E;
    static constexpr int NB = 2 * half + state + tokens <= 160 * 1024 ? 2 : 1;
    static constexpr int sp = NB * half, xp = sp + state, bytes = xp + tokens;
    static constexpr int plane = 2 * kFragSize;  // elements of one plane over tokens
};

constexpr int kNarrowThreads = 2 * kDeltaThreads;

// What a loading wave does for a row's chunks: chunk number i from memory to registers (load, in two pieces) and on to
// LDS (store).  The compute waves' barriers: the first of chunk c after which the other half is free and before which
// chunk c's operands are written, and two more; with one half, a fourth at the chunk's end.  Everyone waits for the
// last at a barrier, so the loads are spread over the time between them: little after the second, where the compute
// waves have the least to do.
template <int NB, int HALF, typename Load, typename Store>
__device__ __forceinline__ void narrow_loader(char* lds, int chunks, Load load, Store store) {
    if (chunks <= 0) return;
    load(0, 0);
    load(0, 1);
    store(lds);
    load(1, 0);
    load(1, 1);
    for (int c = 0; c < chunks; ++c) {
        lds_barrier();
        if (NB == 2) {
            store(lds + (c & 1 ? 0 : HALF));
            load(c + 2, 0);
        }
        lds_barrier();
        lds_barrier();
        if (NB == 2) load(c + 2, 1);
        if (NB == 1 && c + 1 < chunks) {
            lds_barrier();
            store(lds);
            load(c + 2, 0);
            load(c + 2, 1);
        }
    }
}

template <typename T, int DK, int P, Walk W, bool VEC>
__device__ __forceinline__ void narrow_walk(const DeltaParams& p, unsigned tiles, unsigned unit) {
    constexpr int PY = P < 2 ? P : 2, E = (int)sizeof(T), DT = DK / 64, NS = DK / 32;
    using Sh = ChunkShape<T, DK>;
    using Ops = ChunkOperands<T, P>;
    using L = NarrowLds<T, DK, P, (W == kStates ? 0 : PY), (W == kStates ? 2 * P : 2 * P + PY)>;
    extern __shared__ char lds[];
    T *sp = reinterpret_cast<T*>(lds + L::sp), *rp = reinterpret_cast<T*>(lds + L::xp), *us = rp + P * L::plane, *up = us + P * L::plane;

    const unsigned rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const int chunks = (len + kC - 1) / kC;
    int64_t entry = (int64_t)chunk_entry(p, s, first) * p.H + h;

    if (wave_id() >= 4) {
        const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
        const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
        RowShare<T, DK> kr, qr;
        Linear<Ops::a> ops;
        Linear<PY * L::frag_bytes> opa;
        // Behind the row's end the buffers are empty: with no branch around a load the compiler knows how many are in
        // flight and waits for no more than it needs.
        auto load = [&](int c, int piece) {
            const bool in = c < chunks;
            const int64_t t = in ? (int64_t)c * kC : 0, n = in ? min((int64_t)kC, len - t) : 0;
            const char* o = p.w_ops + (entry + (in ? (int64_t)c * p.H : 0)) * Ops::bytes;
            if (piece == 0) {
                kr.load(make_buf(kp + t * p.ldk, n * p.ldk * E), p.ldk, p.dk, VEC);
                return;
            }
            if (W != kStates) qr.load(make_buf(qp + t * p.ldq, n * p.ldq * E), p.ldq, p.dk, VEC);
            ops.load(o, in);
            if (W != kStates) opa.load(o + Ops::a, in);
        };
        auto store = [&](char* to) {
            kr.store(reinterpret_cast<T*>(to + L::ks), nullptr, 0);
            if (W != kStates) qr.store(reinterpret_cast<T*>(to + L::qs), nullptr, 0);
            ops.store(to);
            if (W != kStates) opa.store(to + L::as);
        };
        narrow_loader<L::NB, L::half>(lds, chunks, load, store);
        return;
    }

    __builtin_amdgcn_s_setprio(2);  // before the loading waves of the same unit
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4, tok = wave * 16 + g4;
    const int col = (int)(unit - rh * tiles) * 16 + l16;
    const T* vp = static_cast<const T*>(p.v) + first * p.ldv + (int64_t)h * p.dv;
    T* op = static_cast<T*>(p.o) + (first * p.H + h) * p.dv;
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    // this lane's column: in a state (its wave's keys), in the values and in the output (its wave's tokens)
    const int key = wave * 16 * DT + g4;
    const unsigned soff = col < p.dv ? (unsigned)(key * p.dv + col) * 4u : kNowhere;
    const unsigned voff = col < p.dv ? (unsigned)(tok * p.ldv + col) * E : kNowhere;
    const unsigned ooff = col < p.dv ? (unsigned)(tok * p.H * p.dv + col) * E : kNowhere;
    const int vals = (p.dv + 63) / 64 * 64;

    f32x4 S[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) S[d] = f32x4{0, 0, 0, 0};
    if (p.h0) {
        const Buf b = make_buf(p.h0 + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[d][r] = buf_load<float>(b, soff + (unsigned)((d * 16 + r) * p.dv) * 4u);
    }
    unsigned v[4];
    auto fetch = [&](int c) {  // the values of chunk c
        const bool in = c < chunks;
        const int64_t t = in ? (int64_t)c * kC : 0, n = in ? min((int64_t)kC, len - t) : 0;
        const Buf vb = make_buf(vp + t * p.ldv, n * p.ldv * E);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = buf_load_bits<T>(vb, voff + (unsigned)(r * p.ldv) * E);
    };
    fetch(0);

    for (int c = 0; c < chunks; ++c, entry += p.H) {
        const int64_t t0 = (int64_t)c * kC, n_tok = min((int64_t)kC, len - t0);
        const bool update = c + 1 < chunks || (W != kStates && p.hT);
        const char* half = lds + (L::NB == 2 && (c & 1) ? L::half : 0);
        const ChunkRows* rows = reinterpret_cast<const ChunkRows*>(half);
        const T *ts = reinterpret_cast<const T*>(half + L::ts), *as = reinterpret_cast<const T*>(half + L::as),
                *ks = reinterpret_cast<const T*>(half + L::ks), *qs = reinterpret_cast<const T*>(half + L::qs);
        // the state's parts
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const int td = wave * DT + d;
            if constexpr (W == kStates)
                store_half_both<PY, P, NS>(S[d], sp, td >> 1, td & 1,
                                           reinterpret_cast<T*>(p.w_s) + entry * PY * vals * DK + (int64_t)col * DK + key + d * 16,
                                           (int64_t)vals * DK);
            else
                store_half<P, NS>(S[d], sp, td >> 1, td & 1);
        }
        lds_barrier();
        // X = K S, Y = Q S for this wave's tokens
        f32x4 X[3], Y[3];
        zero3(X);
        zero3(Y);
        const f32x4 be = four(rows->beta + tok), eg = four(rows->eg + tok), rk = four(rows->rk + tok);
        {
            Parts<T, 1> fk[NS], fq[NS];
            Parts<T, P> fs[NS];
#pragma unroll
            for (int kb = 0; kb < NS; ++kb) {
                fs[kb] = load_exchange<P, NS>(sp, kb);
                const int at = (wave * 16 + l16) * Sh::KS + kb * 32 + g4;
                fk[kb].p[0] = load_runs<T>(ks + at);
                if constexpr (W != kStates) fq[kb].p[0] = load_runs<T>(qs + at);
            }
            loads_end();
#pragma unroll
            for (int kb = 0; kb < NS; ++kb) mma_spread<1, P>(fk[kb], fs[kb], X, 0);
            if constexpr (W != kStates)
#pragma unroll
                for (int kb = 0; kb < NS; ++kb)
#pragma unroll
                    for (int q = PY - 1; q >= 0; --q) Y[(2 * kb + q) % 3] = mma(fq[kb].p[0], fs[kb].p[q], Y[(2 * kb + q) % 3]);
        }
        {
            const f32x4 x = gather3(X);
            f32x4 R;
#pragma unroll
            for (int r = 0; r < 4; ++r) R[r] = be[r] * __builtin_fmaf(-(eg[r] * rk[r]), x[r], Io<T>::of_bits(v[r]));
            store_half<P, 2>(R, rp, wave >> 1, wave & 1);
        }
        fetch(c + 1);
        Parts<T, P> ft[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) ft[kb] = load_parts<P>(ts, lower_frag(wave, wave < 2 ? 0 : kb));
        lds_barrier();
        // U = T R
        f32x4 U;
        {
            Parts<T, P> fr[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) fr[kb] = load_exchange<P, 2>(rp, kb);
            loads_end();
            f32x4 u[3];
            zero3(u);
            mma_spread<P, P>(ft[0], fr[0], u, 0);
            if (wave >= 2) mma_spread<P, P>(ft[1], fr[1], u, 0);
            U = gather3(u);
        }
        store_half<P, 2>(U * (four(rows->er + tok) * rk), us, wave >> 1, wave & 1);
        if constexpr (W == kStates)
            store_four<PY>(U, reinterpret_cast<T*>(p.w_u) + entry * PY * vals * kC + (int64_t)col * kC + tok, (int64_t)vals * kC);
        else
            store_half<PY, 2>(U, up, wave >> 1, wave & 1);
        lds_barrier();
        // S = e^(G_C) S + (e^(G_C - G) K)^T U, O = e^G Y + A U
        Parts<T, P> fu[2];
        Parts<T, PY> fa[2], fo[2];
        Parts<T, 1> fk[DT][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            fu[kb] = load_exchange<P, 2>(us, kb);
#pragma unroll
            for (int d = 0; d < DT; ++d) fk[d][kb].p[0] = load_transposed<T>(ks + kb * 32 * Sh::KS + (wave * DT + d) * 16, Sh::KS);
            if constexpr (W != kStates) {
                fa[kb] = load_parts<PY>(as, lower_frag(wave, wave < 2 ? 0 : kb));
                fo[kb] = load_exchange<PY, 2>(up, kb);
            }
        }
        loads_end();
        if (update) {
            const float ec = rows->eg[kC - 1];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                f32x4 x[3];
                zero3(x);
                x[0] = S[d] * ec;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) mma_spread<1, P>(fk[d][kb], fu[kb], x, 0);
                S[d] = gather3(x);
            }
        }
        if constexpr (W != kStates) {
            const f32x4 f = eg * four(rows->rq + tok) * p.scale;
#pragma unroll
            for (int i = 0; i < 3; ++i) Y[i] *= f;
            mma_spread<PY, PY>(fa[0], fo[0], Y, 0);
            if (wave >= 2) mma_spread<PY, PY>(fa[1], fo[1], Y, 0);
            const f32x4 o = gather3(Y);
            const Buf ob = make_buf(op + t0 * p.H * p.dv, n_tok * p.H * p.dv * E);
#pragma unroll
            for (int r = 0; r < 4; ++r) buf_store<T>(ob, ooff + (unsigned)(r * p.H * p.dv) * E, from_f32<T>(o[r]));
        }
        if (L::NB == 1 && c + 1 < chunks) lds_barrier();
    }
    if (W == kStates || !p.hT) return;
    const Buf sb = make_buf(p.hT + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) buf_store<float>(sb, soff + (unsigned)((d * 16 + r) * p.dv) * 4u, S[d][r]);
}

template <typename T, int DK, int P, bool VEC>
__global__ __launch_bounds__(kNarrowThreads, 2) void delta_narrow_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    narrow_walk<T, DK, P, kPrepared, VEC>(p, tiles, die_local(blockIdx.x, units));
}

template <typename T, int DK, int P> hipError_t launch_narrow(const DeltaParams& p, hipStream_t s) {
    constexpr int PY = P < 2 ? P : 2;
    auto kern = p.vec_k ? delta_narrow_kernel<T, DK, P, true> : delta_narrow_kernel<T, DK, P, false>;
    constexpr int bytes = NarrowLds<T, DK, P, PY, 2 * P + PY>::bytes;
    const hipError_t e = allow_lds(kern, bytes);
    if (e != hipSuccess) return e;
    const unsigned tiles = (p.dv + 15) / 16, units = (unsigned)p.rows * p.H * tiles;
    hipLaunchKernelGGL(kern, dim3(units), dim3(kNarrowThreads), bytes, s, p, tiles, units);
    return hipGetLastError();
}

template <typename T, int DK, int P> hipError_t launch_forward(const DeltaParams& p, hipStream_t s) {
    if (!p.w_ops && p.L <= kC && !p.h0 && !p.hT)
        if constexpr (P < 3) return launch_walk<T, DK, P, kSingle>(p, s);  // (three parts only with states)
    if (!p.w_ops) return launch_walk<T, DK, P, kWhole>(p, s);
    const hipError_t e = launch_prepare<T, DK, P>(p, s);
    if (e != hipSuccess) return e;
    return p.narrow ? launch_narrow<T, DK, P>(p, s) : launch_walk<T, DK, P, kPrepared>(p, s);
}

}  // namespace sfm
