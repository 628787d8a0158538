// sfm_delta_api.cpp -- the C ABI of the gated delta rule (declared in include/sfm.h): argument checks and dispatch.
#include "sfm.h"

#include <hip/hip_runtime.h>

#include <cstdlib>

#include "sfm_api_util.h"
#include "sfm_delta.h"

using namespace sfm::api;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Sizes, strides and types every entry point of the rule shares.
sfm_status check_sizes(const char* fn, int64_t rows, int64_t L, int64_t tokens, bool packed, int64_t Hk, int64_t H,
                       int64_t dk, int64_t dv, int io_dtype, int flags, bool back) {
    if (io_dtype != SFM_F32 && io_dtype != SFM_BF16) return fail(SFM_ERR_DTYPE, "%s: io_dtype %d", fn, io_dtype);
    if (flags & ~SFM_DELTA_L2NORM) return fail(SFM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, flags);
    if (!sane(rows, 1 << 24) || !sane(L, 1 << 24) || tokens < 0 || tokens > (1LL << 31) - 1)
        return fail(SFM_ERR_SHAPE, "%s: rows=%lld L=%lld tokens=%lld out of range", fn, (long long)rows, (long long)L,
                    (long long)tokens);
    if (!packed && tokens != rows * L)
        return fail(SFM_ERR_SHAPE, "%s: %lld tokens are not rows=%lld of L=%lld", fn, (long long)tokens,
                    (long long)rows, (long long)L);
    if (!sane(Hk, 4096) || !sane(H, 4096) || H % Hk)
        return fail(SFM_ERR_SHAPE, "%s: %lld value heads over %lld key heads", fn, (long long)H, (long long)Hk);
    if (!sane(dk, sfm::kDeltaMaxK) || !sane(dv, sfm::kDeltaMaxV))
        return fail(SFM_ERR_SHAPE, "%s: head sizes dk=%lld (1 to %d), dv=%lld (1 to %d)", fn, (long long)dk,
                    sfm::kDeltaMaxK, (long long)dv, sfm::kDeltaMaxV);
    const int64_t widest = dk > dv ? dk : dv;
    if (tokens * H > (1LL << 40) / widest) return fail(SFM_ERR_SHAPE, "%s: tensor too large", fn);
    // the largest launches that no plan avoids: the walks, and the backward's by chunk and head (shared heads: four to one)
    const int64_t walks = rows * H * ((dv + 63) / 64) * (back ? 2 : 1), heads = H != Hk && 4 * Hk > H ? 4 * Hk : H;
    if (walks > sfm::kDeltaMaxGroups || (back && sfm::delta_chunk_entries(rows, tokens) * heads > sfm::kDeltaMaxGroups))
        return fail(SFM_ERR_SHAPE, "%s: rows=%lld tokens=%lld with %lld heads are more workgroups than a launch holds", fn,
                    (long long)rows, (long long)tokens, (long long)H);
    return SFM_OK;
}

sfm_status check_inputs(const char* fn, const void* q, const void* k, const void* v, const void* g, const void* beta,
                        int64_t tokens, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int64_t ldq, int64_t ldk,
                        int64_t ldv, int io_dtype) {
    if (tokens > 0 && (!q || !k || !v || !g || !beta))
        return fail(SFM_ERR_NULL, "%s: q, k, v, g and beta are required", fn);
    if (ldq < Hk * dk || ldk < Hk * dk || ldv < H * dv || ldq > (1 << 22) || ldk > (1 << 22) || ldv > (1 << 22))
        return fail(SFM_ERR_SHAPE, "%s: token strides %lld, %lld, %lld below the heads' widths (or too large)", fn,
                    (long long)ldq, (long long)ldk, (long long)ldv);
    const uintptr_t e = io_bytes(io_dtype);
    if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(g, e) || !aligned_to(beta, e))
        return fail(SFM_ERR_ALIGN, "%s: an input is not aligned to its element", fn);
    return SFM_OK;
}

// Rows up to this long go token by token: a chunk costs its 64 tokens whatever is in it, a token its own reads of the
// values and, the first, the state's.  At 256 rows x 16 heads of 64 x 64: 10 us a token against 49 us a chunk in
// bfloat16 (87 us with states, 48 us for four tokens), against 89 us in float32 (39 us for four).
int64_t recurrent_most(int io_dtype, bool state) { return io_dtype == SFM_F32 ? 10 : state ? 7 : 4; }

struct Ranges {
    Range ins[10];
    int n = 0;
    void add(const char* name, const void* p, int64_t bytes) {
        if (p && bytes > 0) ins[n++] = rng(name, p, bytes);
    }
    void add_inputs(const void* q, const void* k, const void* v, const void* g, const void* beta, int64_t tokens,
                    int64_t Hk, int64_t H, int64_t dk, int64_t dv, int64_t ldq, int64_t ldk, int64_t ldv, int e) {
        if (tokens <= 0) return;
        add("q", q, ((tokens - 1) * ldq + Hk * dk) * e);
        add("k", k, ((tokens - 1) * ldk + Hk * dk) * e);
        add("v", v, ((tokens - 1) * ldv + H * dv) * e);
        add("g", g, tokens * H * e);
        add("beta", beta, tokens * H * e);
    }
    const char* hit(const Range& r) const {
        for (int i = 0; i < n; ++i)
            if (overlap(r, ins[i])) return ins[i].name;
        return nullptr;
    }
};

sfm::DeltaParams params(const void* q, const void* k, const void* v, const void* g, const void* beta, int64_t rows,
                        int64_t L, int64_t tokens, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int64_t ldq,
                        int64_t ldk, int64_t ldv, float scale, int flags, int io_dtype) {
    sfm::DeltaParams p{};
    const int e = io_bytes(io_dtype);
    p.q = q, p.k = k, p.v = v, p.g = g, p.beta = beta;
    p.ldq = ldq, p.ldk = ldk, p.ldv = ldv, p.tokens = tokens;
    p.rows = (int)rows, p.L = (int)L, p.Hk = (int)Hk, p.H = (int)H, p.share = (int)(H / Hk), p.dk = (int)dk, p.dv = (int)dv;
    p.scale = scale;
    p.l2norm = flags & SFM_DELTA_L2NORM ? 1 : 0;
    // 16-byte loads of whole rows need every row to start on 16 bytes
    p.vec_k = aligned16(q) && aligned16(k) && dk * e % 16 == 0 && ldq * e % 16 == 0 && ldk * e % 16 == 0;
    p.vec_v = aligned16(v) && dv * e % 16 == 0 && ldv * e % 16 == 0;
    return p;
}

}  // namespace

// The longest row as the plans see it: L, or where L says nothing of it (packed rows, all the tokens or more) at most
// four times their average.  With L all the tokens, planned by this / by L: 1000 rows to 400 tokens, 16 heads of 128:
// 2440 us, no workspace / 3290 us, 1.8 GB; 256 rows to 200 tokens, 8 heads of 64: 77 / 113 us; their backwards 10.9 /
// 15.5 ms, 357 / 460 us.  Against that, one row of 16384 among 200 of 100 (16 heads of 64) or of 50000 among 1000 of 50
// (128) takes 3 times what it does with its length in L: 1960 / 630 us, 7.6 / 2.6 ms.
static int64_t delta_longest(int64_t rows, int64_t L, int64_t tokens) {
    const int64_t four = (4 * tokens + rows - 1) / rows;
    return L < tokens || four >= L ? L : four < 1 ? 1 : four;
}

// Workgroups of 64 value columns that rows of the longest one's length would make of all the tokens: what a launch
// has to fill the card with, and keeps filling it with, also where packed rows differ.
static int64_t delta_units(int64_t L, int64_t tokens, int64_t H, int64_t dv) { return tokens * H * ((dv + 63) / 64) / L; }

// Few such workgroups walk long rows: the chunks' triangular inverses, which need no state, are then made beforehand
// by the whole card (two launches) instead of inside the walk.  Past 256 the other workgroups of a unit hide their
// making and the operands' way through memory costs more than it saves, unless several column tiles share them
// (values wider than keys); with few values the walk with few columns is the faster one for longer.  bfloat16, inside /
// beforehand:
//     1024 tokens, 64 x 64: 114 / 57 us for 128 workgroups, 115 / 90 us for 256, 143 / 167 us for 384;
//     1024 tokens, 128 x 128: 140 / 66 us for 128, 143 / 109 us for 256, 186 / 217 us for 512;
//     1024 tokens, 64 x 128: 142 / 133 us for 512, 182 / 202 us for 768;
//     1024 tokens, 64 x 32: 142 / 131 us for 384, 144 / 182 us for 512 (float32: 273 / 212 us, 276 / 259 us);
//     two chunks, 64 x 64: 18 / 19 us for 128, 17 / 21 us for 256 (float32: 23 / 22 us, 24 / 28 us).
// SFM_DELTA_WALK=whole|prepared overrides (tuning and tests).
int64_t sfm::plan_delta_fwd(int64_t rows, int64_t L, int64_t tokens, int64_t H, int64_t dk, int64_t dv, bool want_state, int io_dtype) {
    L = delta_longest(rows, L, tokens);
    const int64_t chunks = (L + kDeltaChunk - 1) / kDeltaChunk;
    if (chunks < 2) return 0;  // (nothing to walk, whatever the override says)
    if (delta_chunk_entries(rows, tokens) * H > kDeltaMaxGroups) return 0;  // (more than one launch can prepare)
    const int64_t most = chunks < 3 ? 128 : (dv + 63) / 64 > (dk + 63) / 64 ? 512 : dv <= 32 ? 384 : 256;
    bool prepared = delta_units(L, tokens, H, dv) <= most;
    if (const char* e = std::getenv("SFM_DELTA_WALK")) prepared = e[0] == 'p' || (e[0] != 'w' && prepared);
    return prepared ? delta_chunk_entries(rows, tokens) * H * delta_operand_bytes(io_dtype, want_state ? 3 : 2, 2) : 0;
}

// Walks with few columns to a workgroup (delta_narrow.h: 32 with up to 64 keys, else 16) while there are no more of
// them than run at once, two to a unit of bfloat16 with 64 keys; with 128 keys also twice that, two after one another
// being no slower.  The backward has two walks at once.  64 columns / few, 2048 tokens, bfloat16:
//     64 x 64: 142 / 97 us for 256 of them, 215 / 210 us for 512, 338 / 337 us for 768;
//     128 x 128: 172 / 114 us for 512, 194 / 178 us for 768, 214 / 241 us for 1024;
//     backward, 64 x 64: 211 / 180 us for 128, 281 / 285 us for 192; 128 x 128: 274 / 216 us for 256, 414 / 472 us for 512.
// With up to 32 values half of the 64 columns are nobody's, and few are faster at any number: 64 x 32, 1024 tokens, 92 /
// 69 us for 240 rows and heads, 190 / 182 us for 512; backward 281 / 239 us, 545 / 492 us.
// SFM_DELTA_NARROW=0|1 overrides (tuning and tests).
bool sfm::plan_delta_narrow(int64_t rows, int64_t L, int64_t tokens, int64_t H, int64_t dk, int64_t dv, int io_dtype, bool back) {
    L = delta_longest(rows, L, tokens);
    const bool few = dk <= 64;
    const int64_t cols = few ? 32 : 16;
    if (rows * H * ((dv + 31) / 32 * (32 / cols)) * (back ? 4 : 2) > kDeltaMaxGroups) return false;  // (workgroups of 512)
    if (const char* e = std::getenv("SFM_DELTA_NARROW")) return e[0] == '1';
    if (dv <= 32) return true;
    const int64_t groups = tokens * H * ((dv + cols - 1) / cols) / L;
    return groups <= (back ? (few ? 128 : 256) : few && io_dtype == 0 ? 256 : 512);
}

extern "C" {

sfm_status sfm_gated_delta_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
                                float* state, const int32_t* slots, void* o, int64_t rows, int64_t pool, int64_t Hk,
                                int64_t H, int64_t dk, int64_t dv, int64_t ldq, int64_t ldk, int64_t ldv, float scale,
                                int io_dtype, int flags, void* stream) {
    static const char* fn = "sfm_gated_delta_step";
    sfm_status st = check_sizes(fn, rows, 1, rows, false, Hk, H, dk, dv, io_dtype, flags, false);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, q, k, v, g, beta, rows, Hk, H, dk, dv, ldq, ldk, ldv, io_dtype);
    if (st != SFM_OK) return st;
    if (!state || !o) return fail(SFM_ERR_NULL, "%s: state and o are required", fn);
    if (!sane(pool, 1 << 24) || pool * H > (1LL << 40) / (dk * dv))
        return fail(SFM_ERR_SHAPE, "%s: a pool of %lld states", fn, (long long)pool);
    if (!slots && pool < rows)
        return fail(SFM_ERR_SHAPE, "%s: %lld states for %lld rows (no slots)", fn, (long long)pool, (long long)rows);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(state, 4) || !aligned_to(slots, 4) || !aligned_to(o, e))
        return fail(SFM_ERR_ALIGN, "%s: state, slots or o not aligned to its element", fn);
    Ranges in;
    in.add_inputs(q, k, v, g, beta, rows, Hk, H, dk, dv, ldq, ldk, ldv, e);
    in.add("slots", slots, rows * 4);
    const Range rs = rng("state", state, pool * H * dk * dv * 4), ro = rng("o", o, rows * H * dv * e);
    if (const char* n = in.hit(rs)) return fail(SFM_ERR_ALIAS, "%s: state overlaps %s", fn, n);
    if (const char* n = in.hit(ro)) return fail(SFM_ERR_ALIAS, "%s: o overlaps %s", fn, n);
    if (overlap(rs, ro)) return fail(SFM_ERR_ALIAS, "%s: o overlaps state", fn);
    sfm::DeltaParams p = params(q, k, v, g, beta, rows, 1, rows, Hk, H, dk, dv, ldq, ldk, ldv, scale, flags, io_dtype);
    p.h0 = state, p.hT = state, p.slots = slots, p.pool = pool, p.o = o;
    p.vec_s = dv % 4 == 0 && aligned16(state);
    return hip_status(sfm::launch_delta_recurrent(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

sfm_status sfm_gated_delta_fwd_ws_size(int64_t rows, int64_t L, int64_t tokens, int64_t H, int64_t dk, int64_t dv,
                                       int want_state, int io_dtype, int64_t* bytes) {
    static const char* fn = "sfm_gated_delta_fwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, rows, L, tokens, true, 1, H, dk, dv, io_dtype, 0, false);
    if (st != SFM_OK) return st;
    *bytes = sfm::plan_delta_fwd(rows, L, tokens, H, dk, dv, want_state != 0, io_dtype);
    return ok();
}

sfm_status sfm_gated_delta_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* h0, void* o, float* hT, const int32_t* offsets, int64_t rows, int64_t L,
                               int64_t tokens, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int64_t ldq,
                               int64_t ldk, int64_t ldv, float scale, int io_dtype, int flags, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_gated_delta_fwd";
    sfm_status st = check_sizes(fn, rows, L, tokens, offsets != nullptr, Hk, H, dk, dv, io_dtype, flags, false);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, q, k, v, g, beta, tokens, Hk, H, dk, dv, ldq, ldk, ldv, io_dtype);
    if (st != SFM_OK) return st;
    if (tokens > 0 && !o) return fail(SFM_ERR_NULL, "%s: o is required", fn);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(h0, 4) || !aligned_to(hT, 4) || !aligned_to(offsets, 4) || !aligned_to(o, e))
        return fail(SFM_ERR_ALIGN, "%s: h0, hT, offsets or o not aligned to its element", fn);
    int64_t need = 0;
    st = sfm_gated_delta_fwd_ws_size(rows, L, tokens, H, dk, dv, hT != nullptr, io_dtype, &need);
    if (st != SFM_OK) return st;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(SFM_ERR_SHAPE, "%s: workspace of %lld bytes needed, %lld given", fn, (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    if (need > 0 && !aligned16(workspace)) return fail(SFM_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    const int64_t sb = rows * H * dk * dv * 4;
    Ranges in;
    in.add_inputs(q, k, v, g, beta, tokens, Hk, H, dk, dv, ldq, ldk, ldv, e);
    in.add("offsets", offsets, (rows + 1) * 4);
    in.add("h0", h0, sb);
    Ranges out;
    out.add("o", o, tokens * H * dv * e);
    out.add("workspace", workspace, need);
    for (int i = 0; i < out.n; ++i)
        if (const char* n = in.hit(out.ins[i])) return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, out.ins[i].name, n);
    if (out.n == 2 && overlap(out.ins[0], out.ins[1])) return fail(SFM_ERR_ALIAS, "%s: o overlaps workspace", fn);
    if (hT) {
        const Range r = rng("hT", hT, sb);
        const char* n = in.hit(r);
        if (n && !(hT == h0 && n[0] == 'h')) return fail(SFM_ERR_ALIAS, "%s: hT overlaps %s", fn, n);
        if (const char* m = out.hit(r)) return fail(SFM_ERR_ALIAS, "%s: hT overlaps %s", fn, m);
    }
    sfm::DeltaParams p = params(q, k, v, g, beta, rows, L, tokens, Hk, H, dk, dv, ldq, ldk, ldv, scale, flags, io_dtype);
    p.h0 = h0, p.hT = hT, p.offsets = offsets, p.o = o;
    p.w_ops = need > 0 ? static_cast<char*>(workspace) : nullptr;
    p.narrow = sfm::plan_delta_narrow(rows, L, tokens, H, dk, dv, io_dtype, false);
    p.vec_s = dv % 4 == 0 && aligned16(h0) && aligned16(hT);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    if (L <= recurrent_most(io_dtype, h0 || hT)) return hip_status(sfm::launch_delta_recurrent(p, io_dtype, hs), fn);
    return hip_status(io_dtype == SFM_F32 ? sfm::launch_delta_fwd_f32(p, hs) : sfm::launch_delta_fwd_bf16(p, hs), fn);
}

// Workspace regions of the backward, each on 256 bytes.
struct BwdRegions {
    int64_t ops, s, ds, u, dr, dq, dk, bytes;
};

static BwdRegions bwd_regions(int64_t rows, int64_t tokens, int64_t H, bool shared, int64_t dk, int64_t dv, bool want_dh0,
                              int io_dtype) {
    const int64_t e = io_bytes(io_dtype), units = sfm::delta_chunk_entries(rows, tokens) * H;
    const int64_t vals = (dv + 63) / 64 * 64, keys = dk <= 64 ? 64 : 128, planes = io_dtype == SFM_F32 ? 1 : 2;
    BwdRegions r{};
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    r.ops = take(units * sfm::delta_operand_bytes(io_dtype, want_dh0 ? 3 : 2, want_dh0 ? 3 : 2));
    r.s = take(units * planes * vals * keys * e);
    r.ds = take(units * planes * vals * keys * e);
    r.u = take(units * planes * vals * sfm::kDeltaChunk * e);
    r.dr = take(units * planes * vals * sfm::kDeltaChunk * e);
    r.dq = take(shared ? tokens * H * dk * 4 : 0);
    r.dk = take(shared ? tokens * H * dk * 4 : 0);
    r.bytes = at;
    return r;
}

sfm_status sfm_gated_delta_bwd_ws_size(int64_t rows, int64_t L, int64_t tokens, int64_t Hk, int64_t H, int64_t dk,
                                       int64_t dv, int want_dh0, int io_dtype, int64_t* bytes) {
    static const char* fn = "sfm_gated_delta_bwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, rows, L, tokens, true, Hk, H, dk, dv, io_dtype, 0, true);
    if (st != SFM_OK) return st;
    *bytes = bwd_regions(rows, tokens, H, H != Hk, dk, dv, want_dh0 != 0, io_dtype).bytes;
    return ok();
}

sfm_status sfm_gated_delta_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta,
                               const float* h0, const void* dout, const float* dhT, void* dq, void* dk_out,
                               void* dv_out, void* dg, void* dbeta, float* dh0, const int32_t* offsets, int64_t rows,
                               int64_t L, int64_t tokens, int64_t Hk, int64_t H, int64_t dk, int64_t dv, int64_t ldq,
                               int64_t ldk, int64_t ldv, float scale, int io_dtype, int flags, void* workspace,
                               int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_gated_delta_bwd";
    sfm_status st = check_sizes(fn, rows, L, tokens, offsets != nullptr, Hk, H, dk, dv, io_dtype, flags, true);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, q, k, v, g, beta, tokens, Hk, H, dk, dv, ldq, ldk, ldv, io_dtype);
    if (st != SFM_OK) return st;
    if (tokens > 0 && (!dout || !dq || !dk_out || !dv_out || !dg || !dbeta))
        return fail(SFM_ERR_NULL, "%s: dout, dq, dk, dv, dg and dbeta are required", fn);
    const int e = io_bytes(io_dtype);
    for (const void* x : {(const void*)dout, (const void*)dq, (const void*)dk_out, (const void*)dv_out, (const void*)dg,
                          (const void*)dbeta})
        if (!aligned_to(x, e)) return fail(SFM_ERR_ALIGN, "%s: a gradient is not aligned to its element", fn);
    if (!aligned_to(h0, 4) || !aligned_to(dhT, 4) || !aligned_to(dh0, 4) || !aligned_to(offsets, 4))
        return fail(SFM_ERR_ALIGN, "%s: h0, dhT, dh0 or offsets not aligned to its element", fn);
    const BwdRegions w = bwd_regions(rows, tokens, H, H != Hk, dk, dv, dh0 != nullptr, io_dtype);
    if (!workspace || workspace_bytes < w.bytes)
        return fail(SFM_ERR_SHAPE, "%s: workspace of %lld bytes needed, %lld given", fn, (long long)w.bytes,
                    (long long)(workspace ? workspace_bytes : 0));
    if (!aligned16(workspace)) return fail(SFM_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    const int64_t sb = rows * H * dk * dv * 4, kb = tokens * Hk * dk * e, vb = tokens * H * dv * e, gb = tokens * H * e;
    Ranges in, out;
    in.add_inputs(q, k, v, g, beta, tokens, Hk, H, dk, dv, ldq, ldk, ldv, e);
    in.add("offsets", offsets, (rows + 1) * 4);
    in.add("h0", h0, sb);
    in.add("dout", dout, vb);
    in.add("dhT", dhT, sb);
    out.add("dq", dq, kb);
    out.add("dk", dk_out, kb);
    out.add("dv", dv_out, vb);
    out.add("dg", dg, gb);
    out.add("dbeta", dbeta, gb);
    out.add("dh0", dh0, sb);
    out.add("workspace", workspace, w.bytes);
    for (int i = 0; i < out.n; ++i) {
        if (const char* n = in.hit(out.ins[i])) return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, out.ins[i].name, n);
        for (int j = 0; j < i; ++j)
            if (overlap(out.ins[i], out.ins[j]))
                return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, out.ins[i].name, out.ins[j].name);
    }
    sfm::DeltaParams p = params(q, k, v, g, beta, rows, L, tokens, Hk, H, dk, dv, ldq, ldk, ldv, scale, flags, io_dtype);
    char* ws = static_cast<char*>(workspace);
    p.h0 = h0, p.offsets = offsets, p.dout = dout, p.dhT = dhT;
    p.dq = dq, p.dk_ = dk_out, p.dv_ = dv_out, p.dg = dg, p.dbeta = dbeta, p.dh0 = dh0;
    p.w_ops = ws + w.ops, p.w_s = ws + w.s, p.w_ds = ws + w.ds, p.w_u = ws + w.u, p.w_dr = ws + w.dr;
    p.w_dq = reinterpret_cast<float*>(ws + w.dq), p.w_dk = reinterpret_cast<float*>(ws + w.dk);
    p.vec_o = aligned16(dout) && dv * e % 16 == 0;
    p.narrow = sfm::plan_delta_narrow(rows, L, tokens, H, dk, dv, io_dtype, true);
    const hipStream_t hs = static_cast<hipStream_t>(stream);
    return hip_status(io_dtype == SFM_F32 ? sfm::launch_delta_bwd_f32(p, hs) : sfm::launch_delta_bwd_bf16(p, hs), fn);
}

}  // extern "C"
