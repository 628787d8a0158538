// delta_narrow.h -- the walks of delta_fwd.h and delta_bwd.h for few long rows: 16 columns to a workgroup (128 keys)
// or 32 (64 keys).
//
// A row's chunks follow one another, so where there are few (row, head, 64 column) workgroups the time is that of
// one chunk in one of them, and that is a chain: the state's parts, K S, R, U, the state.  Here four waves share the
// columns, each with 32 keys x 16 columns of the state: K S is then summed over keys through LDS (32 KB a chunk,
// against 60 KB were every wave to read the state's parts for tokens of its own), and the state's parts need not pass
// through LDS before it.  Three barriers a chunk.  Four more waves bring K and Q a chunk ahead, and make the output a
// beat behind; their waits are not the chain's.  Issuing a load stops a wave while the unit takes 64 bytes a cycle,
// so the chain's own loads (T's fragments, straight to registers) are spread over the beat with most else to do.
//
// 2 rows x 8192 tokens x 16 heads of 128 x 128: 204 us for 128 chunks, 3500 cycles each, of which the vector units
// are busy 1300 and LDS 1530; 64 columns to a workgroup: 630 us.  What is left is the chain's own latency (2900
// cycles a chunk where 64 workgroups run) and, with all units busy, 76 KB a chunk and unit from the L2 caches: 12
// TB/s over the card.
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
            const bf16x4 v = take_part(x);
            *reinterpret_cast<bf16x4*>(p + q * NF * kFragSize) = v;
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
            const bf16x4 v = take_part(x);
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

constexpr int kNarrowThreads = 2 * kDeltaThreads;

// ---------------------------------------------------------------- the walk
// Wave w of the four that carry the state has keys 32 kw .. + 31 and columns 16 cw .. + 15 of it.
template <int DK> struct NarrowShape {
    static constexpr int KW = DK / 32, CT = 4 / KW, cols = 16 * CT;  // key groups, column tiles
    int kw, cw;
    __device__ __forceinline__ explicit NarrowShape(int wave) : kw(wave % KW), cw(wave / KW) {}
    // the token tiles of R, U and O that a wave has of its columns: CT of them, the rows of the triangle dealt evenly
    __device__ __forceinline__ int tile(int i) const { return i == 0 ? kw : 3 - kw; }
    // whether a lower triangular operand's row tile has two steps of 32 columns
    __device__ __forceinline__ bool two(int i) const { return CT == 2 ? i == 1 : kw >= 2; }
};

// LDS of the walk: two halves for a chunk's row scalars and K, then what the waves hand one another: the state's first
// PS parts, K S's four tiles in KW sums each, R and U, and U for the output.
template <typename T, int DK, int P, int PS> struct WalkNarrowLds {
    using Sh = ChunkShape<T, DK>;
    using N = NarrowShape<DK>;
    static constexpr int E = (int)sizeof(T), frag = kFragSize * E;
    static constexpr int ks = (int)sizeof(ChunkRows), half = ks + Sh::row_bytes;
    static constexpr int sp = 2 * half, xp = sp + PS * 4 * frag, rp = xp + 16 * 1024, us = rp + P * N::CT * 2 * frag,
                         uf = us + P * N::CT * 2 * frag, bytes = uf + (PS ? N::CT * 4 * 1024 : 0);
    static_assert(bytes <= 160 * 1024, "fits a compute unit");
};

// a fragment's parts of this lane into planes of NF fragments
template <int PW, int P, int NF, typename T> __device__ __forceinline__ void store_exchange(const Parts<T, P>& x, T* base, int frag) {
    T* at = base + frag * kFragSize + (threadIdx.x & 63) * 8;
#pragma unroll
    for (int q = 0; q < PW; ++q) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4*>(at + q * NF * kFragSize) = x.p[q].lo;
            *reinterpret_cast<f32x4*>(at + q * NF * kFragSize + 4) = x.p[q].hi;
        } else {
            *reinterpret_cast<bf16x8*>(at + q * NF * kFragSize) = x.p[q].v;
        }
    }
}
// Eight keys of a row as a fragment: here slot j of lane l stands for key 8 (l / 16) + j of a step of 32, so that the
// keys of a lane are neighbours in memory.  From LDS, and from memory: a buffer of rows from the head's first key on,
// zeros behind its end and behind dk.
template <typename T> __device__ __forceinline__ Frag<T> load_eight(const T* p) { return Frag<T>::load(p); }
template <bool VEC, typename T> __device__ __forceinline__ Frag<T> load_eight(const Buf& b, unsigned at, int key, int dk) {
    typedef T vec8 __attribute__((ext_vector_type(8)));
    constexpr int per = 16 / (int)sizeof(T);
    typedef T piece __attribute__((ext_vector_type(per)));
    vec8 x;
#pragma unroll
    for (int i = 0; i < 8; i += VEC ? per : 1) {
        const unsigned to = key + i < dk ? at + (unsigned)i * (unsigned)sizeof(T) : kNowhere;
        if constexpr (VEC) {
            const piece y = buf_load<piece>(b, to);
#pragma unroll
            for (int e = 0; e < per; ++e) x[i + e] = y[e];
        } else {
            x[i] = buf_load<T>(b, to);
        }
    }
    if constexpr (sizeof(T) == 4)
        return Frag<T>{__builtin_shufflevector(x, x, 0, 1, 2, 3), __builtin_shufflevector(x, x, 4, 5, 6, 7)};
    else
        return Frag<T>{x};
}
// Fragment of K's transpose (32 tokens from p's row on) for the same order: row 4 g + j of tile d is key 8 g + 4 d + j.
template <typename T> __device__ __forceinline__ Frag<T> load_eight_transposed(const T* p, int pitch, int d) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    if constexpr (sizeof(T) == 4) {
        const T* at = p + (l16 >> 2) * 8 + d * 4 + (l16 & 3);
        Frag<T> f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.lo[j] = at[(g4 + j) * pitch];
            f.hi[j] = at[(g4 + 16 + j) * pitch];
        }
        return f;
    } else {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
        const T* at = p + (g4 + (l16 >> 2)) * pitch + (l16 & 3) * 8 + d * 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 16 * pitch));
        return Frag<T>{__builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7))};
    }
}
// the first PW of a fragment's parts as planes of a [row][key] array in memory
template <int PW, int P, typename T> __device__ __forceinline__ void store_eight(const Parts<T, P>& x, T* at, int64_t plane) {
#pragma unroll
    for (int q = 0; q < PW; ++q) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<f32x4*>(at + q * plane) = x.p[q].lo;
            *reinterpret_cast<f32x4*>(at + q * plane + 4) = x.p[q].hi;
        } else {
            *reinterpret_cast<bf16x8*>(at + q * plane) = x.p[q].v;
        }
    }
}
// a computed operand's fragment from the workspace
template <int PA, int P, typename T> __device__ __forceinline__ Parts<T, PA> load_parts(const Buf& b, unsigned at, int f, bool there = true) {
    static_assert(PA <= P, "parts kept");
    typedef unsigned word4 __attribute__((ext_vector_type(4)));
    const unsigned to = fresh(there ? at + (unsigned)(f * kFragSize + (threadIdx.x & 63) * 8) * (unsigned)sizeof(T) : kNowhere);
    Parts<T, PA> a;
#pragma unroll
    for (int q = 0; q < PA; ++q) {
        const unsigned o = to + (unsigned)(q * kLowerFrags * kFragSize) * (unsigned)sizeof(T);
        if constexpr (sizeof(T) == 4) {
            a.p[q].lo = __builtin_bit_cast(f32x4, buf_load<word4>(b, o));
            a.p[q].hi = __builtin_bit_cast(f32x4, buf_load<word4>(b, o + 16));
        } else {
            a.p[q].v = __builtin_bit_cast(bf16x8, buf_load<word4>(b, o));
        }
    }
    return a;
}

// The waves' common beat, chunk c: (1) K S in parts and, for the output, the state lie in LDS; (2) R does; (3) U does,
// and so do chunk c + 1's operands.
template <typename T, int DK, int P, Walk W, bool VEC>
__device__ __forceinline__ void narrow_walk(const DeltaParams& p, unsigned tiles, unsigned unit) {
    constexpr int PY = P < 2 ? P : 2, E = (int)sizeof(T), NS = DK / 32;
    using Sh = ChunkShape<T, DK>;
    using Ops = ChunkOperands<T, P, W == kStates ? P : PY>;
    using N = NarrowShape<DK>;
    using L = WalkNarrowLds<T, DK, P, (W == kStates ? 0 : PY)>;
    constexpr int CT = N::CT, KW = N::KW;
    extern __shared__ char lds[];
    const int wave = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    const N my(wave & 3);

    const unsigned rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const int chunks = (len + kC - 1) / kC;
    int64_t entry = (int64_t)chunk_entry(p, s, first) * p.H + h;
    T *sp = reinterpret_cast<T*>(lds + L::sp), *rp = reinterpret_cast<T*>(lds + L::rp), *us = reinterpret_cast<T*>(lds + L::us);
    f32x4 *xp = reinterpret_cast<f32x4*>(lds + L::xp) + lane, *uf = reinterpret_cast<f32x4*>(lds + L::uf) + lane;
    auto half_of = [&](int c) { return lds + (c & 1 ? L::half : 0); };
    const int col = (int)(unit - rh * tiles) * N::cols + my.cw * 16 + l16;

    if (wave >= 4) {  // these bring the row scalars and K, and make the output a beat behind: O = e^G scale Q S + A U
        if (chunks <= 0) return;
        constexpr bool kOut = W != kStates;
        const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
        const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
        T* op = static_cast<T*>(p.o) + (first * p.H + h) * p.dv;
        RowShare<T, DK> kr;
        Linear<(int)sizeof(ChunkRows)> scalars;
        Parts<T, 1> fq[CT][NS];
        Parts<T, PY> fa[CT][2];
        unsigned qoff[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) qoff[i] = (unsigned)((my.tile(i) * 16 + l16) * (int)p.ldq + 2 * g4) * E;
        // Behind the row's end the buffers are empty: with no branch around a load the compiler knows how many are in
        // flight and waits for no more than it needs.
        auto load_k = [&](int c) {
            const bool in = c < chunks;
            const int64_t t = in ? (int64_t)c * kC : 0, n = in ? min((int64_t)kC, len - t) : 0;
            kr.load(make_buf(kp + t * p.ldk, n * p.ldk * E), p.ldk, p.dk, VEC);
            scalars.load(p.w_ops + (entry + (in ? (int64_t)c * p.H : 0)) * Ops::bytes, in);
        };
        auto store_k = [&](char* to) {
            kr.store(reinterpret_cast<T*>(to + L::ks), nullptr, 0);
            scalars.store(to);
        };
        auto load_q = [&](int c) {
            const bool in = c < chunks;
            const int64_t t = in ? (int64_t)c * kC : 0, n = in ? min((int64_t)kC, len - t) : 0;
            const Buf qb = make_buf(qp + t * p.ldq, n * p.ldq * E);
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                const unsigned at = fresh(qoff[i]);
#pragma unroll
                for (int kb = 0; kb < NS; ++kb) fq[i][kb].p[0] = load_eight<VEC, T>(qb, at + kb * 32u * E, kb * 32 + 2 * g4, p.dk);
            }
        };
        auto load_a = [&](int c) {
            const bool in = c < chunks;
            const Buf ob = make_buf(p.w_ops + (entry + (in ? (int64_t)c * p.H : 0)) * Ops::bytes, in ? Ops::bytes : 0);
#pragma unroll
            for (int i = 0; i < CT; ++i)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
                    if (CT == 1 || kb == 0 || i == 1) fa[i][kb] = load_parts<PY, PY, T>(ob, Ops::a, lower_frag(my.tile(i), kb), kb == 0 || my.two(i));
        };
        load_k(0);
        store_k(lds);
        load_k(1);
        if constexpr (kOut) {
            load_q(0);
            load_a(0);
        }
        lds_barrier();
        for (int c = 0; c < chunks; ++c) {
            lds_barrier();
            f32x4 y[CT][3];
            if constexpr (kOut) {
                const ChunkRows* rows = reinterpret_cast<const ChunkRows*>(half_of(c));
                Parts<T, PY> fs[NS];
#pragma unroll
                for (int kb = 0; kb < NS; ++kb) fs[kb] = load_exchange<PY, 4>(sp, my.cw * KW + kb);
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    zero3(y[i]);
#pragma unroll
                    for (int kb = 0; kb < NS; ++kb)
#pragma unroll
                        for (int q = PY - 1; q >= 0; --q) y[i][(2 * kb + q) % 3] = mma(fq[i][kb].p[0], fs[kb].p[q], y[i][(2 * kb + q) % 3]);
                    const int tok = my.tile(i) * 16 + g4;
                    const f32x4 f = four(rows->eg + tok) * four(rows->rq + tok) * p.scale;
#pragma unroll
                    for (int j = 0; j < 3; ++j) y[i][j] *= f;
                }
                load_q(c + 1);
            }
            lds_barrier();
            store_k(half_of(c + 1));
            load_k(c + 2);
            lds_barrier();
            if constexpr (kOut) {
                const int64_t t0 = (int64_t)c * kC, n_tok = min((int64_t)kC, len - t0);
                const Buf ob = make_buf(op + t0 * p.H * p.dv, n_tok * p.H * p.dv * E);
                Parts<T, PY> fu[2];
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) split<PY>(uf[(my.cw * 4 + 2 * kb) * 64], uf[(my.cw * 4 + 2 * kb + 1) * 64], fu[kb]);
#pragma unroll
                for (int i = 0; i < CT; ++i) {
                    mma_spread<PY, PY>(fa[i][0], fu[0], y[i], 0);
                    if (my.two(i)) mma_spread<PY, PY>(fa[i][1], fu[1], y[i], 0);
                    const f32x4 o = gather3(y[i]);
                    const unsigned ooff = col < p.dv ? (unsigned)((my.tile(i) * 16 + g4) * p.H * p.dv + col) * E : kNowhere;
#pragma unroll
                    for (int r = 0; r < 4; ++r) buf_store<T>(ob, ooff + (unsigned)(r * p.H * p.dv) * E, from_f32<T>(o[r]));
                }
                load_a(c + 1);
            }
        }
        return;
    }

    const T* vp = static_cast<const T*>(p.v) + first * p.ldv + (int64_t)h * p.dv;
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    const int key = my.kw * 32 + 2 * g4;
    const unsigned soff = col < p.dv ? (unsigned)(key * p.dv + col) * 4u : kNowhere;
    const int vals = (p.dv + 63) / 64 * 64;

    f32x4 S[2];
#pragma unroll
    for (int d = 0; d < 2; ++d) S[d] = f32x4{0, 0, 0, 0};
    if (p.h0) {
        const Buf b = make_buf(p.h0 + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[d][r] = buf_load<float>(b, soff + (unsigned)((d * 4 + r) * p.dv) * 4u);
    }
    unsigned v[CT][4];
    auto fetch = [&](int c) {  // the values of chunk c
        const bool in = c < chunks;
        const int64_t t = in ? (int64_t)c * kC : 0, n = in ? min((int64_t)kC, len - t) : 0;
        const Buf vb = make_buf(vp + t * p.ldv, n * p.ldv * E);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const unsigned voff = fresh(col < p.dv ? (unsigned)((my.tile(i) * 16 + g4) * p.ldv + col) * E : kNowhere);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[i][r] = buf_load_bits<T>(vb, voff + (unsigned)(r * p.ldv) * E);
        }
    };
    Parts<T, 1> fk[4];  // K's rows, this wave's keys, of the chunk to come
    auto load_k = [&](int c) {
        const T* ks = reinterpret_cast<const T*>(half_of(c) + L::ks) + my.kw * 32 + l16 * Sh::KS + 2 * g4;
#pragma unroll
        for (int t = 0; t < 4; ++t) fk[t].p[0] = load_eight<T>(ks + t * 16 * Sh::KS);
    };
    const int64_t entry0 = entry;
    Parts<T, P> ft[CT][2];  // T's rows of this wave's tokens
    auto load_t = [&](int c, int kb) {
        const bool in = c < chunks;
        const Buf b = make_buf(p.w_ops + (entry0 + (in ? (int64_t)c * p.H : 0)) * Ops::bytes, in ? Ops::bytes : 0);
#pragma unroll
        for (int i = 0; i < CT; ++i)
            if (CT == 1 || kb == 0 || i == 1) ft[i][kb] = load_parts<P, P, T>(b, Ops::t, lower_frag(my.tile(i), kb), kb == 0 || my.two(i));
    };
    if (chunks > 0) {
        load_t(0, 0);
        fetch(0);
        lds_barrier();
        load_k(0);
    }

    for (int c = 0; c < chunks; ++c, entry += p.H) {
        const bool update = c + 1 < chunks || (W != kStates && p.hT);
        const char* half = half_of(c);
        const ChunkRows* rows = reinterpret_cast<const ChunkRows*>(half);
        const T* ks = reinterpret_cast<const T*>(half + L::ks);
        // K S over this wave's keys
        {
            Parts<T, P> fs;
            split<P>(S[0], S[1], fs);
            if constexpr (W != kStates) store_exchange<PY, P, 4>(fs, sp, my.cw * KW + my.kw);
            f32x4 x[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) x[t] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < P; ++q)  // (the first part's products run while the next is taken)
#pragma unroll
                for (int t = 0; t < 4; ++t) x[t] = mma(fk[t].p[0], fs.p[q], x[t]);
#pragma unroll
            for (int t = 0; t < 4; ++t) xp[((my.cw * 4 + t) * KW + my.kw) * 64] = x[t];
            load_t(c, 1);
            if constexpr (W == kStates)
                store_eight<PY>(fs, reinterpret_cast<T*>(p.w_s) + entry * PY * vals * DK + (int64_t)col * DK + key, (int64_t)vals * DK);
        }
        f32x4 be[CT], ek[CT], er[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int tok = my.tile(i) * 16 + g4;
            be[i] = four(rows->beta + tok);
            ek[i] = four(rows->eg + tok) * four(rows->rk + tok);
        }
        lds_barrier();
        // R = beta (V - e^G K S)
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int t = my.tile(i);
            f32x4 x[KW];
#pragma unroll
            for (int k = 0; k < KW; ++k) x[k] = xp[((my.cw * 4 + t) * KW + k) * 64];
            f32x4 sum = x[0] + x[1];
            if constexpr (KW == 4) sum += x[2] + x[3];
            f32x4 R;
#pragma unroll
            for (int r = 0; r < 4; ++r) R[r] = be[i][r] * __builtin_fmaf(-ek[i][r], sum[r], Io<T>::of_bits(v[i][r]));
            store_half<P, CT * 2>(R, rp, my.cw * 2 + (t >> 1), t & 1);
        }
        fetch(c + 1);
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int tok = my.tile(i) * 16 + g4;
            er[i] = four(rows->er + tok) * four(rows->rk + tok);
        }
        lds_barrier();
        // U = T R
        f32x4 U[CT];
        {
            Parts<T, P> fr[2];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) fr[kb] = load_exchange<P, CT * 2>(rp, my.cw * 2 + kb);
            loads_end();
#pragma unroll
            for (int i = 0; i < CT; ++i) {
                f32x4 u[3];
                zero3(u);
                mma_spread<P, P>(ft[i][0], fr[0], u, 0);
                if (my.two(i)) mma_spread<P, P>(ft[i][1], fr[1], u, 0);
                U[i] = gather3(u);
            }
        }
        Parts<T, 1> kt[2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int d = 0; d < 2; ++d) kt[d][kb].p[0] = load_eight_transposed<T>(ks + kb * 32 * Sh::KS + my.kw * 32, Sh::KS, d);
        loads_end();
#pragma unroll
        for (int i = 0; i < CT; ++i) {
            const int t = my.tile(i);
            store_half<P, CT * 2>(U[i] * er[i], us, my.cw * 2 + (t >> 1), t & 1);
            if constexpr (W == kStates)
                store_four<PY>(U[i], reinterpret_cast<T*>(p.w_u) + entry * PY * vals * kC + (int64_t)col * kC + t * 16 + g4, (int64_t)vals * kC);
            else
                uf[(my.cw * 4 + t) * 64] = U[i];
        }
        const float ec = rows->eg[kC - 1];
        lds_barrier();
        // S = e^(G_C) S + (e^(G_C - G) K)^T U
        Parts<T, P> fu[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) fu[kb] = load_exchange<P, CT * 2>(us, my.cw * 2 + kb);
        if (CT == 1) load_k(c + 1);
        loads_end();
        if (update) {
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                f32x4 x[3];
                zero3(x);
                x[0] = S[d] * ec;
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) mma_spread<1, P>(kt[d][kb], fu[kb], x, 0);
                if (d == 0) {  // (spread over this beat: a wave stands still while a load finds no room)
                    loads_end();
                    load_t(c + 1, 0);
                    loads_end();
                }
                S[d] = gather3(x);
            }
        }
        if (CT > 1) {  // (no registers for them before)
            loads_end();
            load_k(c + 1);
        }
    }
    if (W == kStates || !p.hT) return;
    const Buf sb = make_buf(p.hT + sbase, (int64_t)p.dk * p.dv * 4);
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) buf_store<float>(sb, soff + (unsigned)((d * 4 + r) * p.dv) * 4u, S[d][r]);
}

template <typename T, int DK, int P, bool VEC>
__global__ __launch_bounds__(kNarrowThreads, (DK == 64 && sizeof(T) == 2 && VEC ? 4 : 2)) void delta_narrow_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    narrow_walk<T, DK, P, kPrepared, VEC>(p, tiles, row_unit(p, blockIdx.x, units, tiles * p.H, tiles * p.share));
}

template <typename T, int DK, int P> hipError_t launch_narrow(const DeltaParams& p, hipStream_t s) {
    constexpr int PY = P < 2 ? P : 2;
    auto kern = p.vec_k ? delta_narrow_kernel<T, DK, P, true> : delta_narrow_kernel<T, DK, P, false>;
    constexpr int bytes = WalkNarrowLds<T, DK, P, PY>::bytes;
    const hipError_t e = allow_lds(kern, bytes);
    if (e != hipSuccess) return e;
    constexpr unsigned cols = NarrowShape<DK>::cols;
    const unsigned tiles = (p.dv + cols - 1) / cols, units = (unsigned)p.rows * p.H * tiles;
    hipLaunchKernelGGL(kern, dim3(units), dim3(kNarrowThreads), bytes, s, p, tiles, units);
    return hipGetLastError();
}

template <typename T, int DK, int P> hipError_t launch_forward(const DeltaParams& p, hipStream_t s) {
    if (!p.w_ops && p.L <= kC && !p.h0 && !p.hT)
        if constexpr (P < 3) return launch_walk<T, DK, P, kSingle>(p, s);  // (three parts only with states)
    if (!p.w_ops) return launch_walk<T, DK, P, kWhole>(p, s);
    const hipError_t e = launch_prepare<T, DK, P, (P < 2 ? P : 2)>(p, s);  // (A makes the output only)
    if (e != hipSuccess) return e;
    return p.narrow ? launch_narrow<T, DK, P>(p, s) : launch_walk<T, DK, P, kPrepared>(p, s);
}

}  // namespace sfm
