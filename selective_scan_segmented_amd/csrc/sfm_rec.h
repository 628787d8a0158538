// sfm_rec.h -- host/device contract of the gated linear recurrence's kernels.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfm {

// How a call's rows are cut (plan_rec): a workgroup is nr rows x nt chunks of tokens x nc lanes of `lane` channels.
// Rows longer than nt chunks are cut into blocks of that many: one after the other by one workgroup, or (hand) a
// workgroup each, which hand their states on through the workspace.
template <bool BACK> constexpr int kRecChunk = BACK ? 8 : 16;  // tokens to a lane (recurrence.hip)
struct RecPlan {
    int lane, nc, nt, nr, tiles;  // tiles: workgroups side by side over the channels
    int block;                    // tokens to a block
    int hand;                     // threads to a workgroup that hands on, else 0
    int blocks;                   // equal rows: blocks to a row
    int groups;                   // hand: ticket counters to a tile, a power of two
    int subs;                     // hand: runs of 32 lanes to a tile
    int64_t entries;              // hand: blocks of all rows; else: workgroups along the rows
    int64_t launch;               // workgroups
    int64_t bytes_words, bytes;   // workspace: tickets and words; with the backward's parts of dlam
    uint64_t by_tiles;            // 2^40 / tiles, rounded up: n by_tiles / 2^40 is n / tiles for n < 2^24
    float inv_nc, inv_row;        // 1 / nc, 1 / (nc nt)
};

// One call's rows, channels and strides (forward, backward and the step).
struct RecParams {
    const void* x;           // token t, channel d: x + t * ldx + d (elements)
    const void* r;
    const void* i;
    const float* lam;        // [D]
    const float* h0;         // [rows][D] or null (zero); the pool with the step
    void* y;                 // [tokens][D]; read by the backward
    float* hT;               // [rows][D] or null; the pool with the step
    const int32_t* offsets;  // [rows + 1] or null: row s is tokens s * L .. + L - 1
    const int32_t* slots;    // [rows] or null: the state of row s is number slots[s] of `pool`
    int64_t ldx, ldr, ldi, tokens, pool;
    int rows, L, D;
    float c;
    // backward
    const void* dy;          // [tokens][D]
    const float* dhT;        // [rows][D] or null (zero)
    void *dx, *dr, *di;      // [tokens][D]
    float* dlam;             // [D]
    float* dh0;              // [rows][D] or null
    // workspace
    uint32_t* w_tickets;     // [tiles][groups], 64 bytes apart
    uint64_t* w_words;       // [tiles x subs][entries][32 lanes' channels]: what a block makes of a state (rec_block.h)
    float* w_lam;            // [entries][D]: parts of dlam
    RecPlan plan;
};

// Cuts a call; near: the largest token stride is below 2^19 bytes (so that the 8192 tokens of nr rows end below 2^32); lane: channels to a lane (rec_wide, or one).
RecPlan plan_rec(int64_t rows, int64_t L, int64_t tokens, int64_t D, bool packed, bool near, int lane, bool back);
// Largest token strides: the tokens of a block (at most 1024, and no more than a row has) end below 2^31 bytes.
inline int64_t rec_max_stride(int64_t L, int io_bytes) { return (1LL << 31) / ((L < 1024 ? L : 1024) * io_bytes); }
// Channels to a lane: 4 bytes where the sizes, strides and addresses allow it, else one.
inline int rec_wide(int io_dtype) { return io_dtype == 0 ? 1 : 2; }
hipError_t launch_rec_fwd(const RecParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rec_bwd(const RecParams& p, int io_dtype, hipStream_t s);
hipError_t launch_rec_step(const RecParams& p, int io_dtype, hipStream_t s);

}  // namespace sfm
