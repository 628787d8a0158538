// sfm_delta.h -- host/device contract of the gated delta rule's kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfm {

constexpr int kDeltaChunk = 64;        // tokens to a chunk of the chunked kernels
constexpr int kDeltaMaxK = 128;        // largest key head
constexpr int kDeltaMaxV = 256;        // largest value head
constexpr int64_t kDeltaMaxGroups = (1LL << 24) - 1;  // workgroups of 256 to a launch, which holds fewer than 2^32 work items

// One call's rows, heads and strides (forward, backward and the token-by-token form).
struct DeltaParams {
    const void* q;       // token t, key head j: q + t * ldq + j * dk (elements)
    const void* k;
    const void* v;       // token t, head h: v + t * ldv + h * dv
    const void* g;       // [tokens][H]
    const void* beta;
    const float* h0;     // [rows][H][dk][dv] or null (zero states); the pool with slots
    void* o;             // [tokens][H][dv]
    float* hT;           // [rows][H][dk][dv] or null; the pool with slots
    const int32_t* offsets;  // [rows + 1] or null: row s is tokens s * L .. + L - 1
    const int32_t* slots;    // [rows] or null: the state of row s is number slots[s] of `pool` in h0 and hT
    int64_t ldq, ldk, ldv, tokens, pool;
    int rows, L, Hk, H, share, dk, dv;  // share = H / Hk
    float scale;
    int l2norm;
    int vec_k, vec_v;    // q and k (v) rows may be loaded 16 bytes at a time
    int vec_s;           // states likewise
    int vec_o;           // dout likewise
    int narrow;          // sixteen columns to a workgroup of the walks (delta_narrow.h)
    // backward
    const void* dout;    // [tokens][H][dv]
    const float* dhT;    // [rows][H][dk][dv] or null (zero)
    void *dq, *dk_, *dv_, *dg, *dbeta;
    float* dh0;          // or null
    // workspace: for every chunk (chunk_entry) and head
    char* w_ops;         // ChunkOperands
    char *w_s, *w_ds;    // states before the chunk and gradients of those after it, [parts][values][keys]
    char *w_u, *w_dr;    // U and dR, [parts][values][64 tokens]
    float *w_dq, *w_dk;  // [tokens][H][dk]: gradients by value head, where heads share keys
};

// first token and length of row s; offsets outside the tokens (a caller's mistake) are cut to them
__device__ __forceinline__ void delta_row(const DeltaParams& p, int s, int64_t& first, int& len) {
    if (!p.offsets) {
        first = (int64_t)s * p.L;
        len = p.L;
        return;
    }
    int64_t lo = p.offsets[s], hi = p.offsets[s + 1];
    lo = lo < 0 ? 0 : (lo > p.tokens ? p.tokens : lo);
    hi = hi < lo ? lo : (hi > p.tokens ? p.tokens : hi);
    first = lo;
    len = hi - lo > p.L ? p.L : (int)(hi - lo);
}

// unit-length rows: x / sqrt(sum x^2 + this)
constexpr float kDeltaNormEps = 1e-6f;
// Log decays are taken as at least -110: exp of that is already zero in float32 (2^-158), and minus infinity
// (the state's reset) then keeps the differences of a chunk's running sums finite.
constexpr float kDeltaMinGate = -110.0f;

// Workspace of the chunked forward in bytes: 0 where a chunk's T and A are made on the way (delta_fwd.h).
bool plan_delta_narrow(int64_t rows, int64_t L, int64_t tokens, int64_t H, int64_t dk, int64_t dv, int io_dtype, bool back);
int64_t plan_delta_fwd(int64_t rows, int64_t L, int64_t tokens, int64_t H, int64_t dk, int64_t dv, bool want_state, int io_dtype);
// entries of the arrays that hold something for every chunk (chunk_entry): enough for packed and for equal rows
inline int64_t delta_chunk_entries(int64_t rows, int64_t tokens) { return tokens / kDeltaChunk + rows; }
// bytes of a chunk and head's prepared operands (ChunkOperands), with the parts of bfloat16 ones
inline int64_t delta_operand_bytes(int io_dtype, int parts_t, int parts_a) {
    return 8 * kDeltaChunk * 4 + 6 * 64 * 8 * (io_dtype == 0 ? 8 : 2 * (int64_t)(parts_t + parts_a));
}
// chunked forward, one translation unit per io type
hipError_t launch_delta_fwd_f32(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_fwd_bf16(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_bwd_f32(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_bwd_bf16(const DeltaParams& p, hipStream_t s);
hipError_t launch_delta_recurrent(const DeltaParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
