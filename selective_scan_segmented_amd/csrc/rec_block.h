// rec_block.h -- what the forward and the backward of the gated linear recurrence share (gfx950): the place of a
// workgroup among the rows, loads of a chunk, and the states handed from block to block.
#pragma once

#include "rec_gates.h"
#include "sfm_rec.h"

namespace sfm {

// A run of tokens in memory as a buffer: a lane's byte offset, and a token's, which all lanes share, as the other part of
// the address, so that a token costs a lane no address of its own.  (The range check is not used: lanes without a
// token do not load.)
struct RecBuf {
    __amdgpu_buffer_rsrc_t r;
};
template <typename T>
__device__ __forceinline__ RecBuf rec_buf(const void* base, uint32_t token, uint32_t ld, int back = 0) {
    const T* at = static_cast<const T*>(base) + (int64_t)((uint64_t)token * ld) - back;
    return RecBuf{__builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(at), 0, -1, 0x00027000)};
}

// Cache policy of a buffer access: nontemporal (its lines are the first to go).  The inputs are read that way: they are not
// read again here, and their lines leave the outputs' room.  Without / with it, alone: forward, 2 x 8192 x 2048 bfloat16: 69.6 /
// 66.6 us, float32: 120 / 108 us, 512 x 100 x 640: 102 / 92 us; backward, 16 x 4002 x 320 float32: 144 / 142 us, 2 x 8192 x 2048
// bfloat16: 138 / 133 us, 1024 x 32 x 640: 72 / 64 us; 8192 x 2 x 320 (too small to need the room): 25.7 / 26.9 us, back 43.8 /
// 48.8 us.  With a writer of the inputs before and a reader of the outputs behind: 2 x 8192 x 2048 bfloat16: 115 / 109 us, back
// 225 / 215 us, float32: 215 / 194 us; 8192 x 2 x 320: 36.8 / 37.5 us, back 67.8 / 65.6 us.
constexpr int kStreamed = 2;

// `lane` neighbouring channels of a token as they lie in memory: 4 bytes, or one bfloat16 where two are not aligned.
template <typename T, int C> struct RecPack {
    uint32_t v;
    static constexpr bool kHalf = sizeof(T) * C == 2;
    static constexpr uint32_t kMinusInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    __device__ __forceinline__ void load(const RecBuf& b, uint32_t at, uint32_t token) {
        if constexpr (kHalf)
            v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b.r, at, token, kStreamed);
        else
            v = __builtin_amdgcn_raw_buffer_load_b32(b.r, at, token, kStreamed);
    }
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(v);
        return __uint_as_float(j ? v & 0xffff0000u : v << 16);
    }
    template <int POLICY = 0>
    static __device__ __forceinline__ void store(const RecBuf& b, uint32_t at, uint32_t token, const float (&f)[C]) {
        if constexpr (kHalf) {
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (__bf16)f[0]), b.r, at, token, POLICY);
        } else if constexpr (C == 2) {
            typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, bf2{(__bf16)f[0], (__bf16)f[1]}), b.r, at, token, POLICY);
        } else {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), b.r, at, token, POLICY);
        }
    }
};

// first token and length of row s; offsets outside the tokens (a caller's mistake) are cut to them
__device__ __forceinline__ void rec_row(const RecParams& p, int s, uint32_t& first, int& len) {
    if (!p.offsets) {
        first = (uint32_t)s * (uint32_t)p.L;
        len = p.L;
        return;
    }
    int lo = p.offsets[s], hi = p.offsets[s + 1];
    const int tokens = (int)p.tokens;
    lo = lo < 0 ? 0 : (lo > tokens ? tokens : lo);
    hi = hi < lo ? lo : (hi > tokens ? tokens : hi);
    first = (uint32_t)lo;
    len = hi - lo > p.L ? p.L : hi - lo;
}

// Packed rows of several blocks: row s has the entries from first / block + s on, as many as it has blocks and one if it
// has no token, so that entries of rows never meet and tokens / block + rows of them suffice.  The row of an entry is
// the last one that starts at it or before, found by 64 lanes at a time.
__device__ __forceinline__ uint32_t rec_entry(const RecParams& p, int s, int block) {
    int lo = p.offsets[s];
    lo = lo < 0 ? 0 : (lo > (int)p.tokens ? (int)p.tokens : lo);
    return (uint32_t)lo / (uint32_t)block + (uint32_t)s;
}
__device__ __forceinline__ int rec_row_of(const RecParams& p, uint32_t entry, int block, int lane) {
    int lo = 0, hi = p.rows;  // the row is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, s = lo + lane * step;
        const uint64_t m = __ballot(s < hi && rec_entry(p, s, block) <= entry);
        const int k = m ? 63 - __builtin_clzll(m) : 0;  // (entry 0 of row 0 or later: lane 0 is always in)
        lo += k * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    return lo;
}

// A block takes a state h to A h + H.  Its word says so: A's bits (0 <= A <= 1, or NaN) and H's; kRecWhole in A's
// place: H is the state after the block; all ones: nothing yet.  A word is written and read in one piece, so that no
// other order of memory matters.  The words of 32 lanes' channels lie entry by entry, kRecWords to an entry.
template <int C> constexpr int kRecWords = 32 * C;
template <int C> __device__ __forceinline__ uint64_t* rec_words(const RecParams& p, int tile, uint32_t entry, int w) {
    const int64_t run = tile * p.plan.subs + w / kRecWords<C>;
    return p.w_words + (run * p.plan.entries + entry) * kRecWords<C> + w % kRecWords<C>;
}
constexpr uint32_t kRecEmpty = 0xffffffffu, kRecWhole = 0xbf800000u;  // (the latter -1: no A has its sign)

__device__ __forceinline__ void rec_publish(uint64_t* at, uint32_t tag, float h) {
    __hip_atomic_store(at, (uint64_t)__float_as_uint(h) << 32 | tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t rec_factor(float a) { return a == a ? __float_as_uint(a) & 0x7fffffffu : 0x7fc00000u; }

// The state before a block from the words of those before it in the walk (`before` of them, the first the nearest; the
// farthest is always whole in the end).  From the nearest whole one on the words are applied in the order of the walk,
// one after the other as their owners do: the same bits wherever the whole one is found.
// Every wait ends: tickets are drawn in the order of the walk, so the blocks waited for run already or are through, the
// first waits for none, and every workgroup of packed rows says in the end that its word is whole, whatever a caller's
// offsets make of its place.  The limit is far beyond any wait; past it the state is NaN.
// Words to a look, 1 / 4 / 8 / 16: where rows' waits are for tokens that are still on their way, 2 x 8192 x 2048 bfloat16
// forward: 75 / 66 / 74 / 128 us (more ask for more at once, and take registers), 3 x 8192 x 1024: 69 / 60 / 67 / 113 us, back 119 /
// 117 / 133 / 135 us; one long row, which is waited for hop by hop: 1 x 32768 x 320: 85 / 44 / 39 / 41 us, back 168 / 77 / 62 / 59 us,
// 1 x 65536 x 64: 143 / 55 / 41 / 35 us, 1 x 70000 x 320 float32: 186 / 84 / 79 / 86 us.  Four everywhere.
template <bool BACK, int WINDOW, int WORDS>
__device__ __forceinline__ float rec_look_back(const uint64_t* word, int before) {
    const int n = before < WINDOW ? before : WINDOW;
    for (int polls = 0; polls < 1 << 24; ++polls) {
        uint64_t w[WINDOW];
#pragma unroll
        for (int k = 0; k < WINDOW; ++k)
            w[k] = k < n ? __hip_atomic_load(word + (BACK ? k + 1 : -k - 1) * WORDS, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : ~0ull;
        int whole = -1;
        bool open = true;
#pragma unroll
        for (int k = 0; k < WINDOW; ++k) {
            const uint32_t tag = (uint32_t)w[k];
            if (open && tag == kRecWhole) whole = k;
            open = open && tag != kRecWhole && tag != kRecEmpty;
        }
        if (whole >= 0) {
            float h = 0.0f;
#pragma unroll
            for (int k = WINDOW - 1; k >= 0; --k) {
                const float H = __uint_as_float((uint32_t)(w[k] >> 32));
                if (k == whole) h = H;
                if (k < whole) h = __builtin_fmaf(__uint_as_float((uint32_t)w[k]), h, H);
            }
            return h;
        }
        __builtin_amdgcn_s_sleep(1);
    }
    return __uint_as_float(0x7fc00000u);
}

// What a workgroup works on: a block of a row, or nr rows side by side.
struct RecItem {
    int tile;
    int row;            // the (first) row
    int block, blocks;  // of the row: which, and how many (one where it has no token; none: a block that no row has)
    uint32_t entry;     // of w_words and w_lam
    uint32_t first;     // the (first) row's first token
    int len;            // and length
};

// The workgroup's tile and its number among the tile's.
__device__ __forceinline__ void rec_tile(const RecPlan& q, int& tile, uint32_t& rest) {
    rest = (uint32_t)((uint64_t)blockIdx.x * q.by_tiles >> 40);
    tile = (int)(blockIdx.x - rest * (uint32_t)q.tiles);
}

// A row (or rows of one block) that the workgroup walks itself: the walk's first block.
template <bool BACK>
__device__ __forceinline__ RecItem rec_item(const RecParams& p) {
    const int block = p.plan.block;
    RecItem at;
    rec_tile(p.plan, at.tile, at.entry);
    at.row = (int)at.entry * p.plan.nr;
    rec_row(p, at.row, at.first, at.len);
    at.blocks = at.len <= block ? 1 : (int)(((uint32_t)at.len + block - 1) / (uint32_t)block);
    at.block = BACK ? at.blocks - 1 : 0;
    return at;
}

// Rows of several blocks: the next block of the walk, by ticket.  (One barrier.)
template <bool BACK>
__device__ __forceinline__ RecItem rec_draw(const RecParams& p, uint32_t (&shared)[2]) {
    const RecPlan& q = p.plan;
    RecItem at;
    uint32_t rest;
    rec_tile(q, at.tile, rest);
    const uint32_t group = rest & (uint32_t)(q.groups - 1), last = (uint32_t)q.entries - 1;
    const int block = q.block;
    if (threadIdx.x < 64) {  // (a whole wave: rows are searched by 64 lanes)
        uint32_t ticket = 0;
        if (threadIdx.x == 0)
            ticket = __hip_atomic_fetch_add(p.w_tickets + 16 * (uint32_t)(at.tile * q.groups + group), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u;
        ticket = __builtin_amdgcn_readfirstlane(ticket);
        if (p.offsets) shared[1] = rec_row_of(p, BACK ? last - ticket : ticket, block, threadIdx.x);
        shared[0] = ticket;
    }
    lds_barrier();
    const uint32_t ticket = __builtin_amdgcn_readfirstlane(shared[0]);
    if (!p.offsets) {
        // equal rows: those of a group side by side, block after block
        const uint32_t rows = ((uint32_t)p.rows + q.groups - 1) / (uint32_t)q.groups, j = ticket / rows;
        at.row = (int)((ticket - j * rows) * q.groups + group);
        at.block = (int)(BACK ? q.blocks - 1 - j : j);
        at.blocks = at.row < p.rows ? q.blocks : 0;
        at.entry = (uint32_t)(at.row * q.blocks + at.block);
        at.first = (uint32_t)at.row * (uint32_t)p.L;
        at.len = p.L;
    } else {
        at.entry = BACK ? last - ticket : ticket;
        at.row = __builtin_amdgcn_readfirstlane(shared[1]);
        rec_row(p, at.row, at.first, at.len);
        at.blocks = at.len > 0 ? (int)(((uint32_t)at.len + block - 1) / (uint32_t)block) : 1;
        const int j = (int)(at.entry - rec_entry(p, at.row, block));
        at.block = j;
        if (j < 0 || j >= at.blocks) at.block = at.blocks = 0;  // (j < 0: tokens before the first row, or offsets that fall)
    }
    return at;
}

}  // namespace sfm
