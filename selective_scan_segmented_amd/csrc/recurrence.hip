// recurrence.hip -- the gated linear recurrence (gfx950): forward, backward and one token of many requests.
//
//     a_t = exp(-c softplus(lam) sigmoid(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
//
// and with G_t = dy_t + a_{t+1} G_{t+1}, s = sigmoid, m = sqrt(1 - a^2), P = G la (a h_{t-1} - a^2 / m s(i) x):
//
//     dx = G m s(i),  di = dx x (1 - s(i)),  dr = P (1 - s(r)),  dlam = s(lam) / softplus(lam) sum P,  dh0 = a_0 G_0.
//
// Bound by memory: 8 bytes a bfloat16 value forward, 16 backward, against 31 lane operations forward (6 of them at a
// quarter of the rate: 40 us of a SIMD's time beside 52 of memory's at 2 x 8192 x 2048).  So every value is read once and
// a row is spread over as many lanes as it takes to keep the card's loads in flight: a lane holds 16 tokens (backward 8)
// of 4 bytes of channels in registers and finds what they make of a state, h -> A h + H; a lane a channel joins the chunks
// of a block through LDS; then every lane walks its tokens from its own state.  Rows longer than a block hand their states
// on through words in memory (rec_block.h), so that they too are read once.  The backward walks the same way back with
// u_t = a_{t+1} G_{t+1}: a u + a dy; it makes the gates again for its second look at the tokens, from what it holds in
// registers as it lies in memory.
//
// Measured (calls back to back; rate of the bytes that have to move, of 5.1 TB/s that a large copy reaches):
//     forward, bfloat16: 256 x 51 x 640: 14.5 us, 4.6 TB/s (a copy as large 17); 2 x 8192 x 2048: 67 us, 4.0 TB/s, of
//     which 5 are the words' clearing and 8 the waits for states before; 24 rows packed to 2048 x 1024: 60 us, 3.5 TB/s;
//     backward: bfloat16, 256 x 198 x 320: 60 us, 4.3 TB/s, 2 x 8192 x 2048: 133 us, 4.0 TB/s; float32, 16 x 4002 x 320: 142
//     us, 4.6 TB/s (128 us, 5.1 TB/s, where its outputs take the place of the last call's and part of them is still on the card);
//     step: 256 requests x 2048: 3.7 us on the card.
#include "rec_block.h"

namespace sfm {

namespace {

constexpr int kThreads = 512;     // most to a workgroup
constexpr int kFewThreads = 256;  // and to one that walks rows (plan_rec)

// A lane's place in its workgroup: row, chunk (of TT tokens) and channels.
template <int TT> struct Lane {
    int rr, tc, ch, slot;
    uint32_t tok;  // its chunk's first token behind the item's
    bool live;     // has channels
    __device__ __forceinline__ Lane(const RecParams& p, int tile, int C) {
        const RecPlan& q = p.plan;
        rr = 0;
        int rest = (int)threadIdx.x;
        if (q.nr > 1) {
            rr = div_small(rest, q.inv_row);
            rest -= rr * q.nc * q.nt;
        }
        tc = div_small(rest, q.inv_nc);
        const int cl = rest - tc * q.nc;
        ch = (tile * q.nc + cl) * C;
        slot = (int)threadIdx.x * C;  // ([rows][chunks][channels], as the lanes lie)
        tok = (uint32_t)(rr * p.L + tc * TT);  // (several rows: equal ones)
        live = rr < q.nr && tc < q.nt && ch < p.D;
    }
};

// An item's tokens; everything the same for all lanes but n.
struct Chunk {
    uint32_t base;  // its first token, where the workgroup's buffers start
    int rest;       // tokens from there to the block's end (of each row)
    int row, rows;  // its first row, and the rows from there on
    bool first;     // the block is its row's first
    __device__ __forceinline__ Chunk(const RecParams& p, const RecItem& at) {
        const int block = p.plan.block, skip = at.block * block;
        base = at.first + skip;
        rest = at.len - skip < block ? at.len - skip : block;
        row = at.row;
        rows = p.rows - at.row;
        first = skip == 0;
    }
    // tokens of a lane's chunk (as many as are left: 0 or less, none; TT or more, all)
    template <int TT> __device__ __forceinline__ int n(const Lane<TT>& l) const { return l.live && l.rr < rows ? rest - l.tc * TT : 0; }
};

template <typename T, int C, int TT>
__device__ __forceinline__ void load_chunk(RecPack<T, C> (&v)[TT], const void* from, uint32_t ld, const Chunk& c, const Lane<TT>& l, uint32_t none) {
    const RecBuf b = rec_buf<T>(from, c.base, ld);
    const uint32_t at = (l.tok * ld + l.ch) * sizeof(T), token = ld * sizeof(T);
    const int n = c.n(l);
    if (n >= TT) {
#pragma unroll
        for (int t = 0; t < TT; ++t) v[t].load(b, at, t * token);
    } else if (n > 0) {
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            v[t].v = none;
            if (t < n) v[t].load(b, at, t * token);
        }
    }
}

// A wave's priority among those of its unit: waves that ask for tokens go first and those that make gates last, where that
// was seen to help.  Without / with it: forward in bfloat16, 40 x 600 x 1024: 54.2 / 51.1 us, 32 x 4002 x 1024: 247 / 229 us,
// packed to 2048: 60.6 / 60.0 us; backward walked, bfloat16, 256 x 198 x 320: 61.9 / 60.1 us, float32, 32 x 4002 x 1024: 962 /
// 952 us.  Not elsewhere: forward in float32, 2 x 8192 x 2048: 108.1 / 111.9 us, 64 x 198 x 640: 25.7 / 27.3 us; backward handed
// on, 16 x 4002 x 320 float32: 141.8 / 142.1 us, 2 x 8192 x 2048 bfloat16: 134.2 / 134.4 us; nor in rows of one block, 256 x 51
// x 640 forward: 14.3 / 14.3 us.
template <bool ON, int LEVEL> __device__ __forceinline__ void priority() {
    if constexpr (ON) __builtin_amdgcn_s_setprio(LEVEL);
}

// Joins the chunks' (A, H) of [rows][chunks][channels] in LDS: a lane a row and channel.  In their place: the state
// before every chunk.  BACK: chunks from the last to the first.  kept: the state after the block, for the row's next.
template <int C, bool HAND, bool BACK>
__device__ __forceinline__ void join_chunks(const RecParams& p, float2* agg, const RecItem& at, float& kept) {
    const RecPlan& q = p.plan;
    const int width = q.nc * C;
    const float* before = BACK ? p.dhT : p.h0;
    float* after = BACK ? p.dh0 : p.hT;
    const bool starts = at.block == (BACK ? at.blocks - 1 : 0), ends = at.block == (BACK ? 0 : at.blocks - 1);
    for (int m = threadIdx.x; m < q.nr * width; m += blockDim.x) {
        const int rr = q.nr > 1 ? m / width : 0, w = m - rr * width, ch = at.tile * width + w;
        const int64_t s = at.row + rr;
        if (ch >= p.D || s >= p.rows) continue;
        float2* a = agg + rr * q.nt * width + w;
        float h = kept;
        if (starts) h = before ? before[s * p.D + ch] : 0.0f;
        if constexpr (HAND) {
            const bool tells = !ends || p.offsets;  // (packed rows: always, rec_look_back)
            if (!starts || tells) {
                uint64_t* word = rec_words<C>(p, at.tile, at.entry, w);
                float A = 1.0f, H = 0.0f;
#pragma unroll 8
                for (int k = 0; k < q.nt; ++k) {
                    const float2 v = a[(BACK ? q.nt - 1 - k : k) * width];
                    H = __builtin_fmaf(v.x, H, v.y);
                    A *= v.x;
                }
                if (!starts) {
                    if (tells) rec_publish(word, rec_factor(A), H);
                    h = rec_look_back<BACK, 4, kRecWords<C>>(word, BACK ? at.blocks - 1 - at.block : at.block);
                }
                if (tells) rec_publish(word, kRecWhole, __builtin_fmaf(A, h, H));
            }
        }
#pragma unroll 8
        for (int k = 0; k < q.nt; ++k) {
            float2* v = a + (BACK ? q.nt - 1 - k : k) * width;
            const float2 f = *v;
            v->x = h;
            h = __builtin_fmaf(f.x, h, f.y);
        }
        kept = h;
        if (ends && after) after[s * p.D + ch] = h;
    }
}

// A block that no row has: its words say so (packed rows, rec_look_back), and its part of dlam is none.
template <int C, bool BACK>
__device__ __forceinline__ void empty_block(const RecParams& p, const RecItem& at) {
    if (!p.offsets) return;
    const int width = p.plan.nc * C;
    for (int m = threadIdx.x; m < width; m += blockDim.x) {
        rec_publish(rec_words<C>(p, at.tile, at.entry, m), kRecWhole, 0.0f);
        const int ch = at.tile * width + m;
        if (BACK && ch < p.D) p.w_lam[(int64_t)at.entry * p.D + ch] = 0.0f;
    }
}

// FORM: rows of one block, of several that a workgroup walks, or handed on: by workgroups of so many threads.
constexpr int kOne = 0, kWalk = 1;
constexpr int threads_of(int form) { return form > kWalk ? form : form == kWalk ? kFewThreads : kThreads; }  // (at most)

template <typename T, int C, int FORM>
__global__ __launch_bounds__(threads_of(FORM), C == 2 ? (FORM == kFewThreads ? 5 : 4) : 6) void rec_fwd_kernel(const RecParams p) {
    constexpr bool HAND = FORM > kWalk;
    constexpr bool kExact = sizeof(T) == 4;
    constexpr int TT = kRecChunk<false>;
    constexpr bool kUrgent = C == 2 && FORM != kOne;
    // Gates of so many tokens at a time: those behind the row's end are left out, and fewer values are held at once.  All 16 /
    // 4 / 2: one block, 256 x 51 x 640 bfloat16: 15.4 / 14.7 / 14.0 us, 64 x 198 x 640 float32: 25.8 / 25.6 / 25.6 us; handed on,
    // 2 x 8192 x 2048: 67.5 / 66.7 / 66.3 us; walked, 256 x 300 x 512, bfloat16: 71.0 / 66.7 / 74.5 us; float32: 134 / 143 / 148 us.
    constexpr int kGates = HAND ? 2 : FORM == kWalk && C == 1 ? TT : 4;
    // Outputs that stay in the cache for their reader / do not, alone, and between a writer of x and a reader of y: 256 x 51 x 640
    // bfloat16: 16.2 / 14.7 us, 28.0 / 28.0 us; not where rows are handed on, 2 x 8192 x 2048: 66.8 / 64.9 us, 108.6 / 112.1 us,
    // walked, 32 x 600 x 2048: 126.2 / 132.3 us so placed, nor in float32, 256 x 200 x 1024: 172 / 165 us, 305 / 308 us.
    constexpr int kPolicy = FORM == kOne && C == 2 ? kStreamed : 0;
    __shared__ float2 agg_[FORM == kWalk ? 2 : 1][threads_of(FORM) * C];
    __shared__ uint32_t shared[2];
    RecItem at;
    if constexpr (HAND) {
        at = rec_draw<false>(p, shared);
        if (at.blocks == 0) return empty_block<C, false>(p, at);
    } else {
        at = rec_item<false>(p);
    }
    const Lane<TT> l(p, at.tile, C);
    float rate[C], kept = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) rate[j] = l.live ? rec_rate(p.lam[l.ch + j], p.c) : 0.0f;
    for (int turn = 0;; turn ^= 1) {
        float2* agg = agg_[FORM == kWalk ? turn : 0];
        const Chunk c(p, at);
        const int n = c.n(l);
        float a[TT][C], b[TT][C];
        if (l.live) {
            float A[C], H[C];
#pragma unroll
            for (int j = 0; j < C; ++j) A[j] = 1.0f, H[j] = 0.0f;
            if (n > 0) {
                RecPack<T, C> r[TT], i[TT], x[TT];
                priority<kUrgent, 3>();
                load_chunk<T, C, TT>(r, p.r, p.ldr, c, l, RecPack<T, C>::kMinusInf);
                load_chunk<T, C, TT>(i, p.i, p.ldi, c, l, 0);
                load_chunk<T, C, TT>(x, p.x, p.ldx, c, l, 0);
                priority<kUrgent, 0>();
#pragma unroll
                for (int t0 = 0; t0 < TT; t0 += kGates) {
                    if (kGates < TT && t0 >= n) continue;
#pragma unroll
                    for (int t = t0; t < t0 + kGates; ++t)
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            const float la2 = rate[j] * rec_sigmoid<kExact>(r[t].get(j));
                            a[t][j] = exp2_fast(la2);
                            const float m = __builtin_amdgcn_sqrtf(rec_keep2<kExact>(la2, a[t][j]));
                            b[t][j] = m * rec_sigmoid<kExact>(i[t].get(j)) * x[t].get(j);
                            H[j] = __builtin_fmaf(a[t][j], H[j], b[t][j]);
                            A[j] *= a[t][j];
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < C; ++j) agg[l.slot + j] = make_float2(A[j], H[j]);
        }
        lds_barrier();
        priority<kUrgent, 1>();
        join_chunks<C, HAND, false>(p, agg, at, kept);
        lds_barrier();
        if (n > 0) {
            float h[C];
#pragma unroll
            for (int j = 0; j < C; ++j) h[j] = agg[l.slot + j].x;
            const RecBuf y = rec_buf<T>(p.y, c.base, p.D);
            const uint32_t to = (l.tok * (uint32_t)p.D + l.ch) * sizeof(T), token = p.D * sizeof(T);
            auto walk = [&](auto whole) __attribute__((always_inline)) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
#pragma unroll
                    for (int j = 0; j < C; ++j) h[j] = __builtin_fmaf(a[t][j], h[j], b[t][j]);
                    if (decltype(whole)::value || t < n) RecPack<T, C>::template store<kPolicy>(y, to, t * token, h);
                }
            };
            if (n >= TT)
                walk(std::true_type{});
            else
                walk(std::false_type{});
        }
        if (FORM != kWalk || ++at.block >= at.blocks) break;
    }
}

template <typename T, int C, int FORM>
__global__ __launch_bounds__(threads_of(FORM), 4) void rec_bwd_kernel(const RecParams p) {
    constexpr bool HAND = FORM > kWalk;
    constexpr bool kExact = sizeof(T) == 4;
    constexpr int TT = kRecChunk<true>;
    constexpr bool kUrgent = FORM == kWalk;
    constexpr int kGates = FORM == kOne ? 4 : TT;  // (8 / 4: 8192 x 2 x 320 bfloat16: 51.6 / 48.8 us, 256 x 51 x 640: 34.4 / 34.2 us)
    __shared__ float2 agg_[FORM == kWalk ? 2 : 1][threads_of(FORM) * C];
    __shared__ float part[threads_of(FORM) * C];
    __shared__ uint32_t shared[2];
    RecItem at;
    if constexpr (HAND) {
        at = rec_draw<true>(p, shared);
        if (at.blocks == 0) return empty_block<C, true>(p, at);
    } else {
        at = rec_item<true>(p);
    }
    const RecPlan& q = p.plan;
    const Lane<TT> l(p, at.tile, C);
    float rate[C], sum[C], kept = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) rate[j] = l.live ? rec_rate(p.lam[l.ch + j], p.c) : 0.0f, sum[j] = 0.0f;
    for (int turn = 0;; turn ^= 1) {
        float2* agg = agg_[FORM == kWalk ? turn : 0];
        const Chunk c(p, at);
        const int n = c.n(l);
        const bool start = c.first && l.tc == 0;
        RecPack<T, C> g[TT], i[TT], x[TT], y[TT];
        float sr[TT][C];
        if (l.live) {
            float A[C], U[C];
#pragma unroll
            for (int j = 0; j < C; ++j) A[j] = 1.0f, U[j] = 0.0f;
            if (n > 0) {
                RecPack<T, C> r[TT];
                priority<kUrgent, 3>();
                load_chunk<T, C, TT>(r, p.r, p.ldr, c, l, RecPack<T, C>::kMinusInf);
                load_chunk<T, C, TT>(g, p.dy, p.D, c, l, 0);
                load_chunk<T, C, TT>(i, p.i, p.ldi, c, l, 0);
                load_chunk<T, C, TT>(x, p.x, p.ldx, c, l, 0);
                // the states before the tokens: the outputs one earlier
                const RecBuf w = rec_buf<T>(p.y, c.base, p.D, p.D);
                const uint32_t token = p.D * sizeof(T), from = (l.tok * (uint32_t)p.D + l.ch) * sizeof(T);
                if (n >= TT && !start) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) y[t].load(w, from, t * token);
                } else {
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        y[t].v = 0;
                        if (t < n && !(t == 0 && start)) y[t].load(w, from, t * token);
                    }
                }
                priority<kUrgent, 0>();
#pragma unroll
                for (int t0 = TT - kGates; t0 >= 0; t0 -= kGates) {
                    if (kGates < TT && t0 >= n) continue;
#pragma unroll
                    for (int t = t0 + kGates - 1; t >= t0; --t)
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            sr[t][j] = rec_sigmoid<kExact>(r[t].get(j));
                            const float a = exp2_fast(rate[j] * sr[t][j]);
                            U[j] = a * (U[j] + g[t].get(j));
                            A[j] *= a;
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < C; ++j) agg[l.slot + j] = make_float2(A[j], U[j]);
        }
        lds_barrier();
        priority<kUrgent, 1>();
        join_chunks<C, HAND, true>(p, agg, at, kept);
        lds_barrier();
        if (n > 0) {
            float u[C], h0[C];
#pragma unroll
            for (int j = 0; j < C; ++j) {
                u[j] = agg[l.slot + j].x;
                h0[j] = p.h0 && start ? p.h0[(int64_t)(c.row + l.rr) * p.D + l.ch + j] : 0.0f;
            }
            const uint32_t to = (l.tok * (uint32_t)p.D + l.ch) * sizeof(T), token = p.D * sizeof(T);
#pragma unroll
            for (int t = TT - 1; t >= 0; --t) {
                if (t >= n) continue;
                float dx[C], dr[C], di[C];
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const float si = rec_sigmoid<kExact>(i[t].get(j)), xv = x[t].get(j);
                    const float la2 = rate[j] * sr[t][j], la = (rate[j] * kLn2) * sr[t][j];
                    const float a = exp2_fast(la2), em = rec_keep2<kExact>(la2, a);
                    const float rs = __builtin_amdgcn_rsqf(__builtin_fmaxf(em, 0x1p-126f));  // (a = 1: la is 0 beside it)
                    const float G = g[t].get(j) + u[j], before = t == 0 && start ? h0[j] : y[t].get(j);
                    u[j] = a * G;
                    // (u la before all else: 0 where a is, whatever la; and la / m before x, which a shut gate may find large)
                    const float ula = u[j] * la;
                    const float P = __builtin_fmaf(ula, before, -(ula * rs) * (a * (si * xv)));
                    dx[j] = G * (em * rs * si);
                    const float s = dx[j] * xv;
                    di[j] = __builtin_fmaf(-s, si, s);
                    dr[j] = __builtin_fmaf(-P, sr[t][j], P);
                    sum[j] += P;
                }
                RecPack<T, C>::store(rec_buf<T>(p.dx, c.base, p.D), to, t * token, dx);
                RecPack<T, C>::store(rec_buf<T>(p.dr, c.base, p.D), to, t * token, dr);
                RecPack<T, C>::store(rec_buf<T>(p.di, c.base, p.D), to, t * token, di);
            }
        }
        if (FORM != kWalk || --at.block < 0) break;
    }
    if (l.live)
#pragma unroll
        for (int j = 0; j < C; ++j) part[l.slot + j] = sum[j];
    lds_barrier();
    const int width = q.nc * C;
    for (int m = threadIdx.x; m < width; m += blockDim.x) {
        const int ch = at.tile * width + m;
        if (ch >= p.D) continue;
        float all = 0.0f;
#pragma unroll 8
        for (int k = 0; k < q.nr * q.nt; ++k) all += part[k * width + m];
        p.w_lam[(int64_t)at.entry * p.D + ch] = all;
    }
}

// dlam from the workgroups' parts: 16 channels to a workgroup, every 64th part to a lane, eight of them asked for
// together, in 64 bits (1008 parts of 320 channels: 5.4 us, 7.3 where the last few came one by one; 256 parts 4.7).  softplus(lam) ->
// sigmoid(lam) (1 + e^lam / 2) as lam falls: their quotient is 1 in float32 below -17.
__global__ __launch_bounds__(1024) void rec_lam_kernel(const RecParams p) {
    __shared__ double part[64][17];
    const int w = threadIdx.x & 15, g = threadIdx.x >> 4, d = blockIdx.x * 16 + w;
    double sum = 0.0;
    if (d < p.D) {
        const float* v = p.w_lam + d;
        const int64_t n = p.plan.entries;
        for (int64_t k = g; k < n; k += 8 * 64) {
            float f[8];
#pragma unroll
            for (int m = 0; m < 8; ++m) f[m] = v[(k + m * 64 < n ? k + m * 64 : k) * p.D];
#pragma unroll
            for (int m = 0; m < 8; ++m) sum += k + m * 64 < n ? (double)f[m] : 0.0;
        }
    }
    part[g][w] = sum;
    __syncthreads();
    if (g >= 16) return;
    sum = ((part[g][w] + part[g + 16][w]) + part[g + 32][w]) + part[g + 48][w];
    part[g][w] = sum;  // (its own place, read by none but it before the barrier)
    lds_barrier();
    if (g || d >= p.D) return;
    for (int k = 1; k < 16; ++k) sum += part[k][w];
    const float lam = p.lam[d];
    const float ratio = lam < -17.0f ? 1.0f : rec_sigmoid<true>(lam) / (softplus_log2e(lam) * kLn2);
    p.dlam[d] = (float)sum * ratio;
}

// Tickets and words to all ones (2 MB: 5 us, a launch's own time; as long with other stores or more to a lane).
__global__ __launch_bounds__(256) void rec_clear_kernel(uint4* w, int64_t n) {
    const int64_t k = (int64_t)blockIdx.x * 1024 + threadIdx.x;
#pragma unroll
    for (int m = 0; m < 4; ++m)
        if (k + 256 * m < n) w[k + 256 * m] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// A lane a request and channel; a launch's latency (1.9 us alone, 3.7 us at 256 requests x 2048 channels).
template <typename T>
__global__ __launch_bounds__(256) void rec_step_kernel(const RecParams p) {
    constexpr bool kExact = sizeof(T) == 4;
    const int d = blockIdx.y * 256 + threadIdx.x, s = blockIdx.x;
    if (d >= p.D) return;
    const int64_t slot = p.slots ? p.slots[s] : s;
    T* y = static_cast<T*>(p.y) + (int64_t)s * p.D + d;
    if (slot < 0 || slot >= p.pool) {
        *y = from_f32<T>(0.0f);
        return;
    }
    float* state = p.hT + slot * p.D + d;
    const float la2 = rec_rate(p.lam[d], p.c) * rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.r)[s * p.ldr + d]));
    const float a = exp2_fast(la2), m = __builtin_amdgcn_sqrtf(rec_keep2<kExact>(la2, a));
    const float b = m * rec_sigmoid<kExact>(to_f32(static_cast<const T*>(p.i)[s * p.ldi + d])) *
                    to_f32(static_cast<const T*>(p.x)[s * p.ldx + d]);
    const float h = __builtin_fmaf(a, *state, b);
    *state = h;
    *y = from_f32<T>(h);
}

template <typename T, bool BACK>
hipError_t launch_rows(const RecParams& p, hipStream_t s) {
    const RecPlan& q = p.plan;
    if (q.hand) {
        const int64_t n = q.bytes_words / 16;
        hipLaunchKernelGGL(rec_clear_kernel, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, s, reinterpret_cast<uint4*>(p.w_tickets), n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)q.launch), threads((unsigned)(q.nr * q.nt * q.nc + 63) / 64 * 64);  // (whole waves)
    const int form = q.hand ? q.hand : p.L > q.block ? kWalk : kOne;
#define SFM_REC_LAUNCH(C, FORM)                                                       \
    if (q.lane == C && form == FORM) {                                                \
        if constexpr (BACK)                                                           \
            hipLaunchKernelGGL((rec_bwd_kernel<T, C, FORM>), grid, threads, 0, s, p); \
        else                                                                          \
            hipLaunchKernelGGL((rec_fwd_kernel<T, C, FORM>), grid, threads, 0, s, p); \
    }
    SFM_REC_LAUNCH(1, kOne) SFM_REC_LAUNCH(1, kWalk) SFM_REC_LAUNCH(1, kThreads)
    if constexpr (sizeof(T) == 2) { SFM_REC_LAUNCH(2, kOne) SFM_REC_LAUNCH(2, kWalk) SFM_REC_LAUNCH(2, kThreads) }
    if constexpr (sizeof(T) == 2 && !BACK) { SFM_REC_LAUNCH(2, kFewThreads) }
#undef SFM_REC_LAUNCH
    return hipGetLastError();
}

}  // namespace

// Whether rows of several blocks are handed on or walked by a workgroup each.  Handing on costs a launch that clears the
// words (5 us) and a wait a block; walking leaves the card to the rows and tiles there are, and packed rows to the
// longest of them.  32 tiles, walked / handed on:
//     forward, bfloat16, 12 rows of 600: 33 / 33 us, 16 rows: 37 / 43 us, 8 rows of 2400: 98 / 74 us, 16 rows: 131 / 141 us;
//     three blocks (300 tokens), 2 rows: 13 / 16 us, 4 rows: 15 / 16 us, 8 rows: 17 / 17 us;
//     float32, 16 rows of 600: 40 / 43 us, of 2400: 145 / 135 us, of 8000: 492 / 446 us, 24 rows of 2400: 213 / 206 us;
//     backward, bfloat16, 16 rows of 600: 89 / 82 us, of 2400: 311 / 297 us, 20 rows of 600: 102 / 102 us, of 2400: 377 / 369
//     us, 24 rows of 600: 111 / 122 us, of 2400: 415 / 443 us; five blocks (300 tokens), 8 rows: 38 / 27 us, 16 rows: 49 / 52
//     us (the loss is taken); float32, 16 rows of 600: 81 / 77 us, 24 rows: 111 / 119 us, of 300, 12 rows: 43 / 40 us, 16
//     rows: 47 / 47 us.
// Packed, rows of 1 to the length stated, in 16 tiles where no other width is given; forward, and after the semicolon
// backward.  Short ones, walked / handed on:
//     to 300, bfloat16, 16 rows: 16 / 16 us; 36 / 25, 64 rows: 29 / 30; 55 / 57, 128 rows: 44 / 48; 87 / 95; float32, 32 rows:
//     16 / 19; 40 / 34, 64 rows: 25 / 29; 53 / 54, 128 rows: 39 / 49; 76 / 87; bfloat16 x 511 (one channel to a lane), 64 rows:
//     27 / 32; 51 / 60; to 400, 128 rows, bfloat16: 54 / 60; 112 / 120, float32: 52 / 60; 103 / 109; 500 rows x 64 bfloat16: 23 /
//     34; 57 / 47; of 350 to 400, forward, 8 rows, bfloat16: 18 / 14, float32: 16 / 14 (of 250 to 300: 16 / 14 and 13 / 14), 32
//     rows: 27 / 33 and 27 / 32; 48 rows x 333 bfloat16 (528 tiles): 36 / 32 (the loss is taken).
// Even ones (500 to 600): bfloat16, 16 rows: 29 / 26; 63 / 49, 32 rows: 35 / 43; 85 / 84, 64 rows: 68 / 77; 141 / 151; float32,
//     16 rows: 24 / 23; 57 / 47, 32 rows: 35 / 43; 78 / 78, 64 rows: 67 / 74; 139 / 143 (backward, the loss is taken), 200 x 320:
//     105 / 115; 260 / 236.
// Others: to 600, bfloat16, 64 rows: 45 / 46; 103 / 91, 128 rows: 75 / 79; 169 / 159, 256 rows: 138 / 149; 298 / 306; float32, 64
//     rows: 45 / 45; 98 / 83, 128 rows: 72 / 75; 154 / 148, 256 rows: 136 / 142; 299 / 284, 384 rows: 201 / 204; 424 / 415; to 2000,
//     bfloat16, 128 rows: 266 / 242; 564 / 495, 256 rows: 474 / 458; 975 / 946; float32, 256 rows: 469 / 423; 981 / 894; 1500 to
//     2000, 64 rows, bfloat16: 224 / 220; 447 / 448, float32: 216 / 200; 439 / 426.
static bool hands_on(int64_t rows, int64_t L, int64_t tokens, int tiles, int blocks, bool packed, bool narrow, bool back) {
    if (packed) {
        if (L * rows > 4 * tokens) return true;  // (one far longer than the others, or no bound)
        if (L <= 400) return rows * tiles < (back ? 1024 : 256);
        const bool even = 3 * tokens > 2 * rows * L;
        if (even && L <= 1024 && !back) return rows * tiles < 384;
        return rows * tiles < (narrow ? 6144 : even ? 1024 : L <= 1024 ? 2048 : 4096);
    }
    if (back) return rows * tiles < 640;
    return rows * tiles < (narrow && blocks > 8 ? 800 : 512) && blocks > 3;
}

RecPlan plan_rec(int64_t rows, int64_t L, int64_t tokens, int64_t D, bool packed, bool near, int lane, bool back) {
    RecPlan q{};
    q.lane = lane;
    const int lanes = (int)((D + lane - 1) / lane);
    const int chunk = back ? kRecChunk<true> : kRecChunk<false>;
    const int64_t chunks = (L + chunk - 1) / chunk;
    const int least = lanes < 32 ? lanes : 32;  // lanes side by side: 128 bytes where there are so many
    const int chains = (lanes + least - 1) / least;
    // cuts rows for workgroups of so many threads; whether they then are of several blocks
    const auto cut = [&](int threads) {
        const int most = threads / least < 64 ? threads / least : 64;
        const bool several = chunks > (most > 16 ? most : 16);
        q.nt = several ? most : (int)chunks;
        q.blocks = 1;
        if (several && !packed) {  // (equal rows: equal blocks)
            q.blocks = (int)((chunks + most - 1) / most);
            q.nt = (int)((chunks + q.blocks - 1) / q.blocks);
            q.blocks = (int)((chunks + q.nt - 1) / q.nt);
        }
        return several;
    };
    bool several = cut(kFewThreads);
    if (several && hands_on(rows, L, tokens, chains, q.blocks, packed, lane == 1, back)) {
        // Workgroups that hand on: wide ones make fewer blocks to wait for, small ones more waits at once.  256 / 512 threads:
        //     backward, float32: 1 x 70000 x 320: 260 / 168 us, 16 x 4002 x 320: 145 / 145 us, 2 x 8192 x 2048: 246 / 247 us;
        //     backward, bfloat16: 1 x 20000 x 1024: 104 / 89 us, 2 x 8192 x 2048: 135 / 134 us, 24 packed to 2048 x 1024: 120 / 116 us;
        //     forward, float32: 1 x 70000 x 320: 134 / 84 us, 2 x 8192 x 2048: 110 / 108 us;
        //     forward, bfloat16: 1 x 32768 x 320 (5 rows' tiles): 68 / 44 us, 1 x 8192 x 1024 (16): 27 / 24 us, x 2048 (32):
        //     39 / 39 us, 3 x 8192 x 1024 (48): 60 / 66 us, 2 x 8192 x 2048 (64): 67 / 72 us, packed to 2048: 60 / 63 us.
        const int threads = lane == 1 || back || rows * chains <= 32 ? kThreads : kFewThreads;
        several = cut(threads);
        q.hand = several ? threads : 0;
    }
    q.groups = 1;
    // No bound of the rows, or one that few come near, and rows of few tokens on average: handed on as long ones, but by
    // workgroups of 32 or 64 tokens and so many more channels.  Without / with it, no bound: forward (back), bfloat16, 4096 rows
    // to 16 x 2048: 746 / 264 us (1741 / 561), to 100 x 1024: 572 / 433 us (1261 / 935; with 32 tokens 395 and 836); one row of
    // 50000 among 2048 to 16 x 320, float32: 220 / 214 us (371 / 310; with 32 tokens 348 and 417).  With the bound the first two
    // take 112 and 308 us (234 and 824).
    const bool loose = q.hand && packed && lanes > least && L * rows > 4 * tokens && tokens < 100 * rows;
    if (loose) {
        int64_t nt = (tokens < 24 * rows ? 32 : 64) / chunk;
        if (nt < q.hand / lanes) nt = q.hand / lanes;
        if (nt < q.nt) q.nt = (int)nt;
    }
    // Many packed rows of one block, most far shorter than the longest: lanes for the average's chunks (forward), or for no
    // more than a small workgroup's (backward), walk the longer ones.  One block / this: forward, bfloat16, 4096 rows to 100 x
    // 1024: 382 / 309 us, 512 to 250 x 2048: 241 / 217 us; float32, 2048 to 200 x 320: 179 / 189 us (left out); backward,
    // bfloat16, 4096 to 100 x 1024: 897 / 824 us, float32, 2048 to 100 x 320: 258 / 228 us; rows of 90 to 100 x 320: 395 / 433 us.
    if (packed && !several && rows * chains >= 4096 && 3 * tokens <= 2 * rows * L && (back || lane == 2)) {
        int64_t nt = back ? chunks : (tokens / rows + chunk - 1) / chunk;
        if (nt < lane) nt = lane;  // (a lane of the join to a channel)
        if (nt > kFewThreads / least) nt = kFewThreads / least;
        if (nt < chunks) q.nt = (int)nt;
    }
    q.block = q.nt * chunk;
    // one block: as wide as the workgroup allows in whole 128 bytes, down to half that where it leaves fewer lanes idle
    const int budget = q.nt * least > kFewThreads ? kThreads : kFewThreads;
    int nc = loose ? q.hand / q.nt : several ? least : budget / q.nt;
    if (nc >= lanes) {
        nc = lanes;
    } else if (nc >= 32) {
        const int widest = nc / 32 * 32;
        nc = widest;
        for (int n = widest - 32; n >= 32 && 2 * n >= widest; n -= 32)
            if ((lanes + n - 1) / n * n < (lanes + nc - 1) / nc * nc) nc = n;
    }
    q.nc = nc;
    q.tiles = (lanes + nc - 1) / nc;
    q.subs = (nc + 31) / 32;
    q.nr = several || packed || q.tiles > 1 || !near ? 1 : budget / (q.nt * nc);
    if (q.nr > rows) q.nr = (int)rows;
    if (!q.hand) {
        q.entries = (rows + q.nr - 1) / q.nr;
        q.launch = q.entries * q.tiles;
    } else if (packed) {
        q.entries = tokens / q.block + rows;
        q.launch = q.entries * q.tiles;
    } else {
        q.groups = rows < 2 ? 1 : rows < 4 ? 2 : rows < 8 ? 4 : 8;
        q.entries = rows * q.blocks;
        q.launch = (rows + q.groups - 1) / q.groups * q.groups * q.blocks * q.tiles;
    }
    q.bytes_words = q.hand ? (int64_t)q.tiles * q.groups * 64 + q.entries * q.tiles * q.subs * 32 * lane * 8 : 0;
    q.bytes_words = (q.bytes_words + 15) / 16 * 16;
    q.bytes = q.bytes_words + (back ? q.entries * D * 4 : 0);
    q.by_tiles = ((1ULL << 40) + q.tiles - 1) / q.tiles;
    q.inv_nc = 1.0f / (float)q.nc, q.inv_row = 1.0f / (float)(q.nc * q.nt);
    return q;
}

hipError_t launch_rec_fwd(const RecParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_rows<float, false>(p, s) : launch_rows<__bf16, false>(p, s);
}

hipError_t launch_rec_bwd(const RecParams& p, int io_dtype, hipStream_t s) {
    const hipError_t e = io_dtype == 0 ? launch_rows<float, true>(p, s) : launch_rows<__bf16, true>(p, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(rec_lam_kernel, dim3((unsigned)((p.D + 15) / 16)), dim3(1024), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_rec_step(const RecParams& p, int io_dtype, hipStream_t s) {
    const dim3 grid((unsigned)p.rows, (unsigned)((p.D + 255) / 256));
    if (io_dtype == 0)
        hipLaunchKernelGGL(rec_step_kernel<float>, grid, dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL(rec_step_kernel<__bf16>, grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace sfm
