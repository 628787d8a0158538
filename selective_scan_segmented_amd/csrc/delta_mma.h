// delta_mma.h -- matrix-instruction fragments of the gated delta rule's kernels (gfx950).
//
// Every product is built from 16 x 16 output tiles with 32 values of the contraction per step.  A fragment is
// eight contraction values of one row (left operand) or one column (right operand) per lane: lane l holds row or
// column l % 16 and the slots 8 (l / 16) .. + 7 of the 32.  Which contraction index sits in which slot is free as
// long as both operands agree, and it is chosen so that results become operands without leaving their lanes: an
// accumulator tile has column l % 16 and rows 4 (l / 16) .. + 3 in lane l, so slot 8 g + 4 h + j stands for index
// 16 h + 4 g + j, and two accumulator tiles that lie one above the other are, lane by lane, the right operand of
// the next product.
//
// bfloat16 tensors use v_mfma_f32_16x16x32_bf16.  What is computed (states, the chunk's inverse, the updates) is
// float32; as an operand it is a sum of two or three bfloat16 parts (8 bits each: relative error 2^-17 or 2^-25)
// and the products of parts below that size are left out, so results keep float32's grade at the bfloat16 matrix
// rate (2 or 3 instructions against an input operand, 3 or 6 between two computed ones; the float32 instruction
// takes 16 times the bfloat16 one's time a product).  float32 tensors use v_mfma_f32_16x16x4_f32, eight to a step.
#pragma once

#include "sfm_device.h"

namespace sfm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// this wave's number in its workgroup, known to the compiler as one value for all lanes
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Operand loads above stay above: issued together, they are in flight while the instructions between run.
__device__ __forceinline__ void loads_end() { __builtin_amdgcn_sched_barrier(0); }

// ---------------------------------------------------------------- bounded memory
// A run of device memory as a buffer: loads past its end give zero and stores there are dropped, so rows behind the
// end of a chunk and columns behind a head's need no branch (a branch round every load makes them wait in turn).
struct Buf {
    __amdgpu_buffer_rsrc_t r;
};
constexpr unsigned kNowhere = 0x80000000u;  // an offset past every buffer (they end below 2^30, offsets add less)
__device__ __forceinline__ Buf make_buf(const void* p, int64_t bytes) {
    return Buf{__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000)};
}
// The value as one the compiler must take afresh: sums of it with each of a loop's constants are then made where
// they are used, not all kept in registers across the loop.
__device__ __forceinline__ unsigned fresh(unsigned v) {
    asm volatile("" : "+v"(v));
    return v;
}
// one element's bits in a register of its own (neighbours are not packed, which would wait for both), and its value
template <typename T> __device__ __forceinline__ unsigned buf_load_bits(const Buf& b, unsigned at) {
    if constexpr (sizeof(T) == 2)
        return (unsigned)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(b.r, at, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b32(b.r, at, 0, 0);
}
template <typename T> __device__ __forceinline__ T buf_load(const Buf& b, unsigned at) {
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(T, (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(b.r, at, 0, 0));
    else if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(b.r, at, 0, 0));
    else
        return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b128(b.r, at, 0, 0));
}
template <typename T> __device__ __forceinline__ void buf_store(const Buf& b, unsigned at, T v) {
    if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), b.r, at, 0, 0);
    else
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), b.r, at, 0, 0);
}

template <typename T> struct Frag;
template <> struct Frag<__bf16> {
    bf16x8 v;
    static __device__ __forceinline__ Frag load(const __bf16* p) { return Frag{*reinterpret_cast<const bf16x8*>(p)}; }
};
template <> struct Frag<float> {
    f32x4 lo, hi;
    static __device__ __forceinline__ Frag load(const float* p) {
        return Frag{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
    }
};

__device__ __forceinline__ f32x4 mma(const Frag<__bf16>& a, const Frag<__bf16>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma4(f32x4 a, f32x4 b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
    return mma4(a.hi, b.hi, mma4(a.lo, b.lo, c));
}

// Four values rounded to bfloat16, of which x keeps the rounding errors (exact: a float32's is a float32).  They are
// taken back from the pairs as packed: two instructions a value and level, where a conversion apiece would be three.
__device__ __forceinline__ bf16x4 take_part(f32x4& x) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef unsigned word2 __attribute__((ext_vector_type(2)));
    word2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        unsigned u = __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x[2 * i], x[2 * i + 1]}), bf16x2));
        asm("" : "+v"(u));
        w[i] = u;
        x[2 * i] -= __builtin_bit_cast(float, u << 16);
        x[2 * i + 1] -= __builtin_bit_cast(float, u & 0xffff0000u);
    }
    return __builtin_bit_cast(bf16x4, w);
}

// A computed operand: P parts whose sum is the float32 values (one part for float32).
template <typename T, int P> struct Parts {
    Frag<T> p[P];
};

// the parts of eight float32 values in slot order (lo: slots 0..3, hi: slots 4..7 of the lane)
template <int P> __device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Parts<__bf16, P>& out) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const bf16x4 a = take_part(lo), b = take_part(hi);
        out.p[q].v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
}
template <int P> __device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Parts<float, P>& out) {
    out.p[0] = Frag<float>{lo, hi};
}

// Fragment of a [token][key] array whose keys lie in their own order: slots 0..3 and 4..7 of a lane are the runs at
// 4 (l / 16) and 16 further on.
template <typename T> __device__ __forceinline__ Frag<T> load_runs(const T* p) {
    typedef T quad __attribute__((ext_vector_type(4)));
    const quad lo = *reinterpret_cast<const quad*>(p), hi = *reinterpret_cast<const quad*>(p + 16);
    if constexpr (sizeof(T) == 4)
        return Frag<T>{lo, hi};
    else
        return Frag<T>{__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)};
}

// Fragment of the transpose of a [token][key] array: rows are the 16 keys from `keys` on (p points at the array's
// element [32 tokens' first][keys' first]), the contraction runs over 32 tokens.  bfloat16: the LDS read that
// transposes 4 x 16 values among 16 lanes (lane i gives the address of token i / 4, keys 4 (i % 4) .. + 3, and
// receives key i of the four tokens); float32: element by element.
template <typename T> __device__ __forceinline__ Frag<T> load_transposed(const T* p, int pitch) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    if constexpr (sizeof(T) == 4) {
        Frag<T> f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.lo[j] = p[(g4 + j) * pitch + l16];
            f.hi[j] = p[(g4 + 16 + j) * pitch + l16];
        }
        return f;
    } else {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4* lds_ptr;
        const T* at = p + (g4 + (l16 >> 2)) * pitch + (l16 & 3) * 4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 16 * pitch));
        return Frag<T>{__builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7))};
    }
}

// Computed operands [64][64], lower triangle of tiles: fragment by fragment, 64 lanes x 8 slots each, so a lane
// writes what the same lane of any wave reads.  Row tile rt, step kb of 32 columns:
__device__ __forceinline__ constexpr int lower_frag(int rt, int kb) { return rt < 2 ? rt : 2 * rt - 2 + kb; }
constexpr int kLowerFrags = 6;
constexpr int kFragSize = 64 * 8;

// tile (rt, tj)'s four values of this lane (row l % 16, columns 4 (l / 16) .. + 3) into P planes
template <int P, typename T> __device__ __forceinline__ void store_tile(f32x4 x, T* base, int rt, int tj) {
    const int lane = threadIdx.x & 63;
    T* p = base + lower_frag(rt, tj >> 1) * kFragSize + lane * 8 + (tj & 1) * 4;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(p) = x;
    } else {
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const bf16x4 v = take_part(x);
            *reinterpret_cast<bf16x4*>(p + q * kLowerFrags * kFragSize) = v;
        }
    }
}

// the same to memory: byte `at` of a buffer
template <int P, typename T> __device__ __forceinline__ void store_tile(f32x4 x, const Buf& b, unsigned at, int rt, int tj) {
    const int lane = threadIdx.x & 63;
    at += (unsigned)(lower_frag(rt, tj >> 1) * kFragSize + (tj & 1) * 4) * (unsigned)sizeof(T) + (unsigned)lane * 8u * (unsigned)sizeof(T);
    if constexpr (sizeof(T) == 4) {
        typedef unsigned word4 __attribute__((ext_vector_type(4)));
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(word4, x), b.r, at, 0, 0);
    } else {
        typedef unsigned word2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const bf16x4 v = take_part(x);
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(word2, v), b.r, at + q * kLowerFrags * kFragSize * 2, 0, 0);
        }
    }
}

// c[rt] += the step kb of 32 columns of a lower triangular operand (its fragments' parts) times b: the products of parts
// that are not below the last part of the finer operand, smallest first; those of like size follow one another, so that
// no accumulator waits for itself
template <int PA, int PB, typename T>
__device__ __forceinline__ void mma_lower(const Parts<T, PA> (&a)[kLowerFrags], const Parts<T, PB>& b, int kb, f32x4 (&c)[4]) {
    constexpr int top = PA > PB ? PA : PB;
#pragma unroll
    for (int p = PA - 1; p >= 0; --p)
#pragma unroll
        for (int q = PB - 1; q >= 0; --q)
            if (p + q < top)
#pragma unroll
                for (int rt = 2 * kb; rt < 4; ++rt) c[rt] = mma(a[lower_frag(rt, kb)].p[p], b.p[q], c[rt]);
}

// likewise with the transpose of a lower triangular operand (upper_frag's order)
__device__ __forceinline__ constexpr int upper_frag(int jt, int kb) { return jt < 2 ? 2 * jt + kb : jt + 2; }
template <int PA, int PB, typename T>
__device__ __forceinline__ void mma_upper(const Parts<T, PA> (&a)[kLowerFrags], const Parts<T, PB>& b, int kb, f32x4 (&c)[4]) {
    constexpr int top = PA > PB ? PA : PB;
#pragma unroll
    for (int p = PA - 1; p >= 0; --p)
#pragma unroll
        for (int q = PB - 1; q >= 0; --q)
            if (p + q < top)
#pragma unroll
                for (int jt = 0; jt < 2 * kb + 2; ++jt) c[jt] = mma(a[upper_frag(jt, kb)].p[p], b.p[q], c[jt]);
}

// parts of fragment `f` of a computed operand
template <int P, typename T> __device__ __forceinline__ Parts<T, P> load_parts(const T* base, int f) {
    const int lane = threadIdx.x & 63;
    Parts<T, P> a;
#pragma unroll
    for (int q = 0; q < P; ++q) a.p[q] = Frag<T>::load(base + (q * kLowerFrags + f) * kFragSize + lane * 8);
    return a;
}

// The same of the operand's transpose: row tile jt, contraction over its rows 32 kb .. + 31; row tiles above the
// diagonal (below jt) are zero.
template <int P, typename T> __device__ __forceinline__ Parts<T, P> load_parts_transposed(const T* base, int jt, int kb) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = (lane >> 4) * 4;
    Parts<T, P> a;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const T* plane = base + q * kLowerFrags * kFragSize + (jt & 1) * 4;
        if constexpr (sizeof(T) == 4) {
            // column l16 of the tile lies with lanes 16 (l16 / 4) + row
            auto get = [&](int it) {
                f32x4 v = {0, 0, 0, 0};
                if (it >= jt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = plane[lower_frag(it, jt >> 1) * kFragSize + ((l16 >> 2) * 16 + g4 + j) * 8 + (l16 & 3)];
                return v;
            };
            a.p[q] = Frag<T>{get(2 * kb), get(2 * kb + 1)};
        } else {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            auto get = [&](int it) {
                s16x4 v = {0, 0, 0, 0};
                if (it >= jt)
                    v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_ptr)(plane + lower_frag(it, jt >> 1) * kFragSize + ((l16 & 3) * 16 + g4 + (l16 >> 2)) * 8));
                return v;
            };
            a.p[q].v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(get(2 * kb), get(2 * kb + 1), 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
    return a;
}

// the first PW of a fragment's parts as planes of a [row][16-aligned run] array in memory: slots 0..3 go to `at`,
// 4..7 to `at` + 16 elements (the next tile's rows)
template <int PW, int P, typename T> __device__ __forceinline__ void store_planes(const Parts<T, P>& x, T* at, int64_t plane) {
    typedef T quad __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int q = 0; q < PW; ++q) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<quad*>(at + q * plane) = x.p[q].lo;
            *reinterpret_cast<quad*>(at + q * plane + 16) = x.p[q].hi;
        } else {
            *reinterpret_cast<quad*>(at + q * plane) = __builtin_shufflevector(x.p[q].v, x.p[q].v, 0, 1, 2, 3);
            *reinterpret_cast<quad*>(at + q * plane + 16) = __builtin_shufflevector(x.p[q].v, x.p[q].v, 4, 5, 6, 7);
        }
    }
}

}  // namespace sfm
