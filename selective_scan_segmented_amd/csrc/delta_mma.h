// delta_mma.h -- matrix-instruction fragments of the gated delta rule's kernels (gfx950).
//
// Every product is built from 16 x 16 output tiles with 32 values of the contraction per step.  A fragment is
// eight contraction values of one row (left operand) or one column (right operand) per lane: lane l holds row or
// column l % 16 and the slots 8 (l / 16) .. + 7 of the 32.  Which contraction index sits in which slot is free as
// long as both operands agree, and it is chosen so that results become operands without leaving their lanes: an
// accumulator tile has column l % 16 and rows 4 (l / 16) .. + 3 in lane l, so slot 8 g + 4 h + j stands for index
// 16 h + 4 g + j, and two accumulator tiles that lie one above the other are, lane by lane, the right operand of
// the next product (slot_of below).
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

// slot of contraction index i within its block of 32 (and of the 4-aligned run it starts, if i % 4 == 0)
__device__ __forceinline__ constexpr int slot_of(int i) {
    return (i & ~31) | (((i >> 2) & 3) << 3) | (((i >> 4) & 1) << 2) | (i & 3);
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

// A computed operand: P parts whose sum is the float32 values (one part for float32).
template <typename T, int P> struct Parts {
    Frag<T> p[P];
};

// the parts of eight float32 values in slot order (lo: slots 0..3, hi: slots 4..7 of the lane)
template <int P> __device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Parts<__bf16, P>& out) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            out.p[q].v[j] = (__bf16)lo[j];
            out.p[q].v[4 + j] = (__bf16)hi[j];
        }
        if (q + 1 < P) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // exact: the rounding error of a float32 is a float32
                lo[j] -= (float)out.p[q].v[j];
                hi[j] -= (float)out.p[q].v[4 + j];
            }
        }
    }
}
template <int P> __device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Parts<float, P>& out) {
    out.p[0] = Frag<float>{lo, hi};
}

// four values into P planes of an LDS operand (plane stride `plane` elements)
template <int P> __device__ __forceinline__ void store_parts(f32x4 x, __bf16* p, int plane) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
        bf16x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = (__bf16)x[j];
            x[j] -= (float)v[j];
        }
        *reinterpret_cast<bf16x4*>(p + q * plane) = v;
    }
}
template <int P> __device__ __forceinline__ void store_parts(f32x4 x, float* p, int) {
    *reinterpret_cast<f32x4*>(p) = x;
}

// c[n] += a b[n] for NC column tiles, a in PA planes of an LDS operand, b in PB parts: the products of parts that
// are not below the last part of the finer operand, smallest first
template <int PA, int PB, int NC, typename T>
__device__ __forceinline__ void mma_columns(const T* a, int plane, const Parts<T, PB> (&b)[NC], f32x4 (&c)[NC]) {
    constexpr int top = PA > PB ? PA : PB;
#pragma unroll
    for (int p = PA - 1; p >= 0; --p) {
        const Frag<T> fa = Frag<T>::load(a + p * plane);
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
            for (int q = PB - 1; q >= 0; --q)
                if (p + q < top) c[n] = mma(fa, b[n].p[q], c[n]);
    }
}

}  // namespace sfm
