// delta_fwd.h -- the walk over a row's chunks: the gated delta rule's forward, and the states that its backward needs
// (kernels; one translation unit per io type).
//
// A workgroup takes one (row, head) and 64 columns of its values, 16 to a wave, and walks the row's chunks; the
// state's columns stay in the wave's accumulators (float32) all the way.  S0, R and U pass from product to product
// inside a lane (delta_mma.h), so waves meet only over K, Q, T and A in LDS.
//
// What bounds it: one chunk takes a workgroup some 7 us with its triangles made on the way (18000 cycles, half of them
// waiting: float32 substitutions, LDS, barriers) and 3.8 us without; the matrix unit is busy 1900 cycles of them with 64
// keys.  Other workgroups of the unit fill the gaps, three of them (four for rows of one chunk, where T takes the place
// of K and Q): 256 x 51 tokens x 10 heads of 64 x 64 in 32 us (67 MB, 2.1 TB/s; 2560 workgroups in 1024 places, so the
// third round is half empty), 1024 workgroups of 1024 tokens in 273 us (294 with two).
#pragma once

#include "delta_chunk.h"

namespace sfm {

// kWhole: T and A of a chunk are made on the way (rows of few chunks, or enough rows to fill the card while some
// workgroups do that).  kPrepared: they come from the preparing kernel.  kStates: likewise, and instead of outputs
// the states before the chunks and U are written down, for the backward.  kSingle: kWhole for rows of one chunk that
// begin and end without a state, which leaves R = beta V, U = T R, O = A U.
enum Walk { kWhole, kPrepared, kStates, kSingle };

// P: parts of T and A.  SINGLE: T takes the place of K and Q, which a chunk without states needs no more by then.
template <typename T, int DK, int P, bool SINGLE = false> struct WalkLds {
    using Sh = ChunkShape<T, DK>;
    static constexpr int frag_bytes = kLowerFrags * kFragSize * (int)sizeof(T);
    static constexpr int rows = 0;
    static constexpr int as = (int)sizeof(ChunkRows) + (SINGLE ? 0 : P * frag_bytes);  // (M before A)
    static constexpr int ks = as + (P * frag_bytes > kBytesM ? P * frag_bytes : kBytesM);
    static constexpr int qs = ks + Sh::row_bytes;
    static constexpr int bytes = qs + Sh::row_bytes;
    static constexpr int ts = SINGLE ? ks : (int)sizeof(ChunkRows);  // (T, A: as ChunkOperands has them)
    static_assert(!SINGLE || P * frag_bytes <= 2 * Sh::row_bytes, "T's place");
    static constexpr int fit = 160 * 1024 / bytes, most = SINGLE && sizeof(T) == 2 ? 4 : SINGLE ? 3 : 2;
    static constexpr int groups = fit < 1 ? 1 : fit < most ? fit : most;  // workgroups to a compute unit
};

template <typename T, int DK, int P, Walk W>
__device__ __forceinline__ void walk(const DeltaParams& p, unsigned tiles, unsigned unit) {
    using Sh = ChunkShape<T, DK>;
    using L = WalkLds<T, DK, P, W == kSingle>;
    constexpr int PY = P < 2 ? P : 2;  // parts that only the outputs see: their type's rounding is far above the third
    using Ops = ChunkOperands<T, P, W == kStates ? P : PY>;
    constexpr int E = (int)sizeof(T);
    constexpr bool kOnTheWay = W == kWhole || W == kSingle;
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs),
      *as = reinterpret_cast<T*>(lds + L::as), *ts = reinterpret_cast<T*>(lds + L::ts);

    const unsigned rh = unit / tiles;
    const int s = (int)(rh / (unsigned)p.H), h = (int)(rh - (unsigned)s * p.H), hk = (int)((unsigned)h / (unsigned)p.share);
    const int lane = threadIdx.x & 63, wave = wave_id(), l16 = lane & 15, g4 = (lane >> 4) * 4;
    const int col0 = (int)(unit - rh * tiles) * 64 + wave * 16, col = col0 + l16;
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    const T* qp = static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk;
    const T* kp = static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk;
    const T* vp = static_cast<const T*>(p.v) + first * p.ldv + (int64_t)h * p.dv;
    const T* gp = static_cast<const T*>(p.g) + first * p.H + h;
    const T* bp = static_cast<const T*>(p.beta) + first * p.H + h;
    T* op = static_cast<T*>(p.o) + (first * p.H + h) * p.dv;
    const int64_t sbase = (int64_t)rh * (p.dk * p.dv);
    // this lane's column in a state, in the values and in the output
    // this lane's place in rows of `ld` elements: its column, rows 4 (l / 16) on (taken afresh: see fresh)
    auto place = [&](int64_t ld, unsigned size) {
        const unsigned l = fresh(threadIdx.x);
        const int c = col0 + (int)(l & 15);
        return c < p.dv ? (unsigned)((int)(l >> 4 & 3) * 4 * (int)ld + c) * size : kNowhere;
    };
    int64_t entry = (int64_t)chunk_entry(p, s, first) * p.H + h;
    const int vals = (int)tiles * 64;  // values in the workspace: whole tiles

    f32x4 S[DK / 16];
#pragma unroll
    for (int d = 0; d < DK / 16; ++d) S[d] = f32x4{0, 0, 0, 0};
    if (W != kSingle && p.h0) {
        const Buf b = make_buf(p.h0 + sbase, (int64_t)p.dk * p.dv * 4);
        const unsigned at = place(p.dv, 4);
#pragma unroll
        for (int d = 0; d < DK / 16; ++d)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[d][r] = buf_load<float>(b, at + (unsigned)((d * 16 + r) * p.dv) * 4u);
    }
    bool zero = W == kSingle || !p.h0;  // the state is zero: its products are left out

    RowShare<T, DK> kr, qr;
    ChunkGates gates;
    Linear<Ops::a> ops;                // row scalars and T
    Linear<PY * L::frag_bytes> opa;    // A
    unsigned v[4][4];                  // values' bits
    auto fetch_v = [&](int64_t t0) {
        const int64_t n = min((int64_t)kC, len - t0);
        const Buf vb = make_buf(vp + t0 * p.ldv, n * p.ldv * E);
        const unsigned at = place(p.ldv, E);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[rt][r] = buf_load_bits<T>(vb, at + (unsigned)((rt * 16 + r) * p.ldv) * E);
    };
    auto fetch = [&](int64_t t0) {
        const int64_t n = min((int64_t)kC, len - t0);
        if (kOnTheWay) gates.load(gp + t0 * p.H, bp + t0 * p.H, p.H, (int)n);
        kr.load(make_buf(kp + t0 * p.ldk, n * p.ldk * E), p.ldk, p.dk, p.vec_k);
        if (W != kStates) qr.load(make_buf(qp + t0 * p.ldq, n * p.ldq * E), p.ldq, p.dk, p.vec_k);
        if (W == kPrepared || W == kStates) {
            const char* o = p.w_ops + entry * Ops::bytes;
            ops.load(o);
            if (W == kPrepared) opa.load(o + Ops::a);
        }
        if (!kOnTheWay) fetch_v(t0);
    };
    if (!kOnTheWay && len > 0) fetch(0);  // ahead of its use by a chunk

    for (int64_t t0 = 0; t0 < len; t0 += kC) {
        const int64_t n_tok = min((int64_t)kC, len - t0);
        const int64_t here = entry;
        entry += p.H;
        f32x4 X[4], Y[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) X[rt] = Y[rt] = f32x4{0, 0, 0, 0};
        // X = K S, Y = Q S; then R = beta (V - e^G X) in X's place
        auto state_products = [&] {
            if (W == kStates || (W != kSingle && !zero)) {
                Frag<T> fk[2][4], fq[2][4];
                auto load = [&](int kb) {
                    const int base = (int)fresh((unsigned)(l16 * Sh::KS + g4));
#pragma unroll
                    for (int rt = 0; rt < 4; ++rt) {
                        const int at = base + rt * 16 * Sh::KS + kb * 32;
                        fk[kb & 1][rt] = load_runs<T>(ks + at);
                        if constexpr (W != kStates) fq[kb & 1][rt] = load_runs<T>(qs + at);
                    }
                };
                constexpr int ahead = kOnTheWay && (DK == 128 || (P == 2 && sizeof(T) == 2)) ? 0 : 1;  // (registers for two workgroups to a unit)
                if (ahead) load(0);
#pragma unroll
                for (int kb = 0; kb < DK / 32; ++kb) {
                    if (kb + ahead < DK / 32) load(kb + ahead);
                    loads_end();
                    Parts<T, P> sp;
                    split<P>(S[2 * kb], S[2 * kb + 1], sp);
                    if constexpr (W == kStates)
                        store_planes<PY>(sp, reinterpret_cast<T*>(p.w_s) + here * PY * vals * DK + (int64_t)col * DK + kb * 32 + g4,
                                        (int64_t)vals * DK);
#pragma unroll
                    for (int q = P - 1; q >= 0; --q)
#pragma unroll
                        for (int rt = 0; rt < 4; ++rt) {
                            X[rt] = mma(fk[kb & 1][rt], sp.p[q], X[rt]);
                            if constexpr (W != kStates)
                                if (q < PY) Y[rt] = mma(fq[kb & 1][rt], sp.p[q], Y[rt]);
                        }
                }
            }
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
                const f32x4 be = four(rows->beta + rt * 16 + g4), f = four(rows->eg + rt * 16 + g4) * four(rows->rk + rt * 16 + g4);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    X[rt][r] = be[r] * (W == kSingle ? Io<T>::of_bits(v[rt][r]) : __builtin_fmaf(-f[r], X[rt][r], Io<T>::of_bits(v[rt][r])));
            }
        };
        if (kOnTheWay) fetch(t0);  // (registers that other workgroups on the unit can use better)
        lds_barrier();  // the chunk before is done with LDS
        if constexpr (kOnTheWay) {
            build_chunk<T, DK, P, PY>(kr, qr, gates, p, rows, ks, qs, as, ts, [&] { fetch_v(t0); }, state_products);
        } else {
            kr.store(ks, nullptr, 0);
            ops.store(lds);
            if (W == kPrepared) {
                qr.store(qs, nullptr, 0);
                opa.store(lds + L::as);
            }
            lds_barrier();
            state_products();
            if (t0 + kC < len) fetch(t0 + kC);
        }
        f32x4 U[4];
        {
            Parts<T, P> tp[kLowerFrags], rp[2];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) tp[lower_frag(rt, 0)] = load_parts<P>(ts, lower_frag(rt, 0));
            loads_end();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) split<P>(X[2 * kb], X[2 * kb + 1], rp[kb]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) U[rt] = f32x4{0, 0, 0, 0};
            mma_lower<P, P>(tp, rp[0], 0, U);
#pragma unroll
            for (int rt = 2; rt < 4; ++rt) tp[lower_frag(rt, 1)] = load_parts<P>(ts, lower_frag(rt, 1));
            mma_lower<P, P>(tp, rp[1], 1, U);
        }
        if constexpr (W == kStates) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                Parts<T, PY> up;
                split<PY>(U[2 * kb], U[2 * kb + 1], up);
                store_planes<PY>(up, reinterpret_cast<T*>(p.w_u) + here * PY * vals * kC + (int64_t)col * kC + kb * 32 + g4, (int64_t)vals * kC);
            }
        } else {
            Parts<T, PY> ap[kLowerFrags], up[2];
            if (W == kWhole) loads_end();  // (T's registers first)
#pragma unroll
            for (int f = 0; f < kLowerFrags; ++f) ap[f] = load_parts<PY>(as, f);
            loads_end();
#pragma unroll
            for (int rt = 0; rt < 4 && W != kSingle; ++rt) Y[rt] *= four(rows->eg + rt * 16 + g4) * four(rows->rq + rt * 16 + g4) * p.scale;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) split<PY>(U[2 * kb], U[2 * kb + 1], up[kb]);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) mma_lower<PY, PY>(ap, up[kb], kb, Y);
            const Buf ob = make_buf(op + t0 * p.H * p.dv, n_tok * p.H * p.dv * E);
            const unsigned at = place((int64_t)p.H * p.dv, E);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    buf_store<T>(ob, at + (unsigned)((rt * 16 + r) * p.H * p.dv) * E, from_f32<T>(Y[rt][r]));
        }
        zero = false;
        if (W == kSingle || (t0 + kC >= len && (W == kStates || !p.hT))) break;  // nobody asks for the state after the last chunk
        const float ec = rows->eg[kC - 1];
        Parts<T, P> up[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            const int r0 = kb * 32 + g4;
            split<P>(U[2 * kb] * (four(rows->er + r0) * four(rows->rk + r0)),
                     U[2 * kb + 1] * (four(rows->er + r0 + 16) * four(rows->rk + r0 + 16)), up[kb]);
        }
#pragma unroll
        for (int d = 0; d < DK / 16; ++d) S[d] *= ec;
        constexpr int kHalf = DK / 32;  // key tiles to a group
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            Frag<T> f[kHalf][2];
#pragma unroll
            for (int d = 0; d < kHalf; ++d)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb) f[d][kb] = load_transposed<T>(ks + kb * 32 * Sh::KS + (half * kHalf + d) * 16, Sh::KS);
            loads_end();
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int q = P - 1; q >= 0; --q)
#pragma unroll
                    for (int d = 0; d < kHalf; ++d) S[half * kHalf + d] = mma(f[d][kb], up[kb].p[q], S[half * kHalf + d]);
        }
    }
    if (W == kStates || W == kSingle || !p.hT) return;
    const Buf sb = make_buf(p.hT + sbase, (int64_t)p.dk * p.dv * 4);
    const unsigned at = place(p.dv, 4);
#pragma unroll
    for (int d = 0; d < DK / 16; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r) buf_store<float>(sb, at + (unsigned)((d * 16 + r) * p.dv) * 4u, S[d][r]);
}

template <typename T, int DK, int P, Walk W>
__global__ __launch_bounds__(kDeltaThreads, (W == kWhole && DK == 64 && P == 2 && sizeof(T) == 2 ? 3 : W != kPrepared || DK == 64 ? WalkLds<T, DK, P, W == kSingle>::groups : 1)) void delta_walk_kernel(const DeltaParams p, unsigned tiles, unsigned units) {
    walk<T, DK, P, W>(p, tiles, row_unit(p, blockIdx.x, units, tiles * p.H, tiles * p.share));
}

// T, A and the row scalars of every chunk and head, a workgroup to each.  T and A go from registers to memory.
template <typename T, int DK> struct PrepareLds {
    static constexpr int rows = 0, mt = (int)sizeof(ChunkRows), ks = mt + kBytesM, qs = ks + ChunkShape<T, DK>::row_bytes,
                         bytes = qs + ChunkShape<T, DK>::row_bytes;
    static constexpr int groups = 160 * 1024 / bytes < 3 ? 160 * 1024 / bytes : 3;
};
// Bound by that latency too (the chunk's 18000 cycles, three to a unit), and by the write: 26 to 32 KB to a chunk and
// head.  ALL: every value head of a key head by one workgroup, K K^T and Q K^T made once (2 x 8192 tokens, 16 heads of
// 128 over 8: 53 us, 60 with a workgroup to each).
template <typename T, int DK, int P, int PA, bool ALL>
__global__ __launch_bounds__(kDeltaThreads, (PrepareLds<T, DK>::groups))
void delta_prepare_kernel(const DeltaParams p, unsigned entries, unsigned units) {
    using L = PrepareLds<T, DK>;
    using Ops = ChunkOperands<T, P, PA>;
    constexpr int E = (int)sizeof(T);
    extern __shared__ char lds[];
    ChunkRows* rows = reinterpret_cast<ChunkRows*>(lds + L::rows);
    T *ks = reinterpret_cast<T*>(lds + L::ks), *qs = reinterpret_cast<T*>(lds + L::qs);
    const unsigned heads = ALL ? p.share : 1, groups = (unsigned)p.H / heads,
                   unit = row_unit(p, blockIdx.x, units, entries / (unsigned)p.rows * groups, p.share / heads), entry = unit / groups;
    const int h = (int)((unit - entry * groups) * heads), hk = (int)((unsigned)h / (unsigned)p.share);
    ChunkAt at;
    if (!chunk_at(p, entry, at)) return;
    const int64_t n = min((int64_t)kC, at.len - at.t0), first = at.first + at.t0;
    const T *gp = static_cast<const T*>(p.g) + first * p.H + h, *bp = static_cast<const T*>(p.beta) + first * p.H + h;
    ChunkGates gates;
    gates.load(gp, bp, p.H, (int)n);
    RowShare<T, DK> kr, qr;
    kr.load(make_buf(static_cast<const T*>(p.k) + first * p.ldk + (int64_t)hk * p.dk, n * p.ldk * E), p.ldk, p.dk, p.vec_k);
    qr.load(make_buf(static_cast<const T*>(p.q) + first * p.ldq + (int64_t)hk * p.dk, n * p.ldq * E), p.ldq, p.dk, p.vec_k);
    char* o = p.w_ops + ((int64_t)entry * p.H + h) * Ops::bytes;
    float* mt = reinterpret_cast<float*>(lds + L::mt);
    f32x4 c[5], a[3], t[4];
    start_chunk<T, DK>(kr, qr, gates, p, rows, ks, qs, c);
    for (unsigned j = 0;; o += Ops::bytes) {
        const Buf ob = make_buf(o, Ops::bytes);
        const bool more = ++j < heads;
        if (more) gates.load(gp + j, bp + j, p.H, (int)n);
        finish_chunk(c, p, rows, mt, a, t, [&] {
            each_a(a, [&](f32x4 x, int rt, int tj) { store_tile<PA, T>(x, ob, Ops::a, rt, tj); });
            if (threadIdx.x < sizeof(ChunkRows) / 16)
                reinterpret_cast<uint4*>(o)[threadIdx.x] = reinterpret_cast<const uint4*>(lds)[threadIdx.x];
        });
        if (more && wave_id() == 0) gates.store(rows);  // (done with the head's; the first rows of T are the shortest)
        each_t(t, [&](f32x4 x, int rt, int tj) { store_tile<P, T>(x, ob, Ops::t, rt, tj); });
        if (!more) return;
        lds_barrier();
    }
}

static_assert(ChunkOperands<float, 1>::bytes == 8 * kC * 4 + 2 * 6 * 64 * 8 * 4 &&
              ChunkOperands<__bf16, 3, 2>::bytes == 8 * kC * 4 + 6 * 64 * 8 * 2 * 5, "delta_operand_bytes");

// dynamic LDS above the default limit has to be asked for
template <typename K> hipError_t allow_lds(K kern, int bytes) {
    if (bytes <= 64 * 1024) return hipSuccess;
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int DK, int P, Walk W> hipError_t launch_walk(const DeltaParams& p, hipStream_t s) {
    auto kern = delta_walk_kernel<T, DK, P, W>;
    constexpr int bytes = WalkLds<T, DK, P, W == kSingle>::bytes;
    const hipError_t e = allow_lds(kern, bytes);
    if (e != hipSuccess) return e;
    const unsigned tiles = (p.dv + 63) / 64, units = (unsigned)p.rows * p.H * tiles;
    hipLaunchKernelGGL(kern, dim3(units), dim3(kDeltaThreads), bytes, s, p, tiles, units);
    return hipGetLastError();
}

// The entries that hold a chunk, or may: launches of a workgroup to each are of this size.  Packed rows: by their
// tokens, since L only bounds the longest (256 rows of 200 tokens or fewer, 8 heads of 64, L all their tokens: 113 us
// forward, 790 with a workgroup to every row and chunk of L; the backward 460, 2093).
inline unsigned launch_entries(const DeltaParams& p) {
    return p.offsets ? (unsigned)delta_chunk_entries(p.rows, p.tokens) : (unsigned)p.rows * (unsigned)((p.L + kC - 1) / kC);
}

template <typename T, int DK, int P, int PA> hipError_t launch_prepare(const DeltaParams& p, hipStream_t s) {
    const unsigned entries = launch_entries(p), groups = entries * p.Hk;
    const bool all = p.share > 1 && groups >= 256;  // (where that leaves every compute unit one)
    auto kern = all ? delta_prepare_kernel<T, DK, P, PA, true> : delta_prepare_kernel<T, DK, P, PA, false>;
    constexpr int bytes = PrepareLds<T, DK>::bytes;
    const hipError_t e = allow_lds(kern, bytes);
    if (e != hipSuccess) return e;
    const unsigned units = all ? groups : groups * p.share;
    hipLaunchKernelGGL(kern, dim3(units), dim3(kDeltaThreads), bytes, s, p, entries, units);
    return hipGetLastError();
}

}  // namespace sfm
