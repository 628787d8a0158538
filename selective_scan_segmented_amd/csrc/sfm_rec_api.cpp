// sfm_rec_api.cpp -- the C ABI of the gated linear recurrence (declared in include/sfm.h): argument checks and dispatch.
#include "sfm.h"

#include <hip/hip_runtime.h>

#include <cstring>
#include <initializer_list>

#include "sfm_api_util.h"
#include "sfm_rec.h"

using namespace sfm::api;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sfm_status check_sizes(const char* fn, int64_t rows, int64_t L, int64_t tokens, bool packed, int64_t D, int io_dtype) {
    if (io_dtype != SFM_F32 && io_dtype != SFM_BF16) return fail(SFM_ERR_DTYPE, "%s: io_dtype %d", fn, io_dtype);
    constexpr int64_t most = (1LL << 31) - 1;  // (a bound of all the tokens is one, whatever the rows' lengths)
    if (!sane(rows, 1 << 24) || !sane(L, most) || tokens < 0 || tokens > most || !sane(D, 1 << 16))
        return fail(SFM_ERR_SHAPE, "%s: rows=%lld L=%lld tokens=%lld D=%lld out of range", fn, (long long)rows,
                    (long long)L, (long long)tokens, (long long)D);
    if (!packed && tokens != rows * L)
        return fail(SFM_ERR_SHAPE, "%s: %lld tokens are not rows=%lld of L=%lld", fn, (long long)tokens,
                    (long long)rows, (long long)L);
    // a launch holds fewer than 2^32 work items (the step's: 256 channels of a row to a workgroup; the rows': plan)
    if (rows * ((D + 255) / 256) >= 1 << 24)
        return fail(SFM_ERR_SHAPE, "%s: rows=%lld of %lld channels are more workgroups than a launch holds", fn,
                    (long long)rows, (long long)D);
    return SFM_OK;
}

// The workspace of a call, wide or near or not (which its tensors' places and strides decide); -1: more than a launch holds.
int64_t need_of(int64_t rows, int64_t L, int64_t tokens, int64_t D, bool packed, int io_dtype, bool back) {
    int64_t need = 0;
    for (int lane : {1, sfm::rec_wide(io_dtype)}) {
        if (D % lane) continue;
        for (bool near : {false, true}) {
            const sfm::RecPlan q = sfm::plan_rec(rows, L, tokens, D, packed, near, lane, back);
            const int64_t threads = (q.nr * q.nt * q.nc + 63) / 64 * 64;
            if (q.launch >= 1LL << 24 || q.launch * threads >= 1LL << 32) return -1;
            if (q.bytes > need) need = q.bytes;
        }
    }
    return need;
}

// The size queries do not say whether rows are packed: the larger of both.
int64_t need_of_either(int64_t rows, int64_t L, int64_t tokens, int64_t D, int io_dtype, bool back) {
    const int64_t a = need_of(rows, L, tokens, D, true, io_dtype, back);
    const int64_t b = tokens == rows * L ? need_of(rows, L, tokens, D, false, io_dtype, back) : 0;
    return a < 0 || b < 0 ? -1 : a > b ? a : b;
}

sfm_status too_large(const char* fn, int64_t rows, int64_t tokens, int64_t D) {
    return fail(SFM_ERR_SHAPE, "%s: rows=%lld of %lld tokens and %lld channels are more workgroups than a launch holds", fn,
                (long long)rows, (long long)tokens, (long long)D);
}

// Cuts the call and gives it its workspace.
void take_plan(sfm::RecParams& p, bool wide, int io_dtype, bool back, void* workspace) {
    int64_t most = p.D;
    for (int64_t ld : {p.ldx, p.ldr, p.ldi}) most = ld > most ? ld : most;
    const bool near = most * io_bytes(io_dtype) < 1 << 19;
    p.plan = sfm::plan_rec(p.rows, p.L, p.tokens, p.D, p.offsets != nullptr, near, wide ? sfm::rec_wide(io_dtype) : 1, back);
    char* at = static_cast<char*>(workspace);
    p.w_tickets = reinterpret_cast<uint32_t*>(at);
    p.w_words = reinterpret_cast<uint64_t*>(at + (int64_t)p.plan.tiles * p.plan.groups * 64);
    p.w_lam = reinterpret_cast<float*>(at + p.plan.bytes_words);
}

sfm_status check_inputs(const char* fn, const void* x, const void* r, const void* i, const float* lam, int64_t tokens,
                        int64_t D, int64_t ldx, int64_t ldr, int64_t ldi, int64_t most, float c, int io_dtype) {
    if (!lam || (tokens > 0 && (!x || !r || !i))) return fail(SFM_ERR_NULL, "%s: x, r, i and lam are required", fn);
    for (int64_t ld : {ldx, ldr, ldi})
        if (ld < D || ld > most)
            return fail(SFM_ERR_SHAPE, "%s: token strides %lld, %lld, %lld below D=%lld or above %lld", fn,
                        (long long)ldx, (long long)ldr, (long long)ldi, (long long)D, (long long)most);
    if (!(c > 0.0f && c <= 1e6f)) return fail(SFM_ERR_SHAPE, "%s: c=%g", fn, (double)c);
    const uintptr_t e = io_bytes(io_dtype);
    if (!aligned_to(x, e) || !aligned_to(r, e) || !aligned_to(i, e) || !aligned_to(lam, 4))
        return fail(SFM_ERR_ALIGN, "%s: an input is not aligned to its element", fn);
    return SFM_OK;
}

// Whether every token's channels can be taken 4 bytes at a time.
bool wide_tokens(std::initializer_list<const void*> tensors, std::initializer_list<int64_t> strides, int io_dtype) {
    for (const void* t : tensors)
        if (!aligned_to(t, 4)) return false;
    for (int64_t ld : strides)
        if (ld % sfm::rec_wide(io_dtype)) return false;
    return true;
}

struct Ranges {
    Range of[10];
    int n = 0;
    void add(const char* name, const void* p, int64_t bytes) {
        if (p && bytes > 0) of[n++] = rng(name, p, bytes);
    }
    void add_inputs(const void* x, const void* r, const void* i, const float* lam, int64_t tokens, int64_t D, int64_t ldx,
                    int64_t ldr, int64_t ldi, int e) {
        add("lam", lam, D * 4);
        if (tokens <= 0) return;
        add("x", x, ((tokens - 1) * ldx + D) * e);
        add("r", r, ((tokens - 1) * ldr + D) * e);
        add("i", i, ((tokens - 1) * ldi + D) * e);
    }
};

// No output on an input or on another output, but hT on the whole of h0: that input by its name, since other inputs can
// have the same place and size (lam, with one row).
sfm_status check_ranges(const char* fn, const Ranges& in, const Ranges& out) {
    const auto in_place = [](const Range& o, const Range& i) {
        return !strcmp(o.name, "hT") && !strcmp(i.name, "h0") && o.lo == i.lo && o.hi == i.hi;
    };
    for (int j = 0; j < out.n; ++j) {
        const Range& o = out.of[j];
        for (int k = 0; k < in.n; ++k)
            if (overlap(o, in.of[k]) && !in_place(o, in.of[k]))
                return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, o.name, in.of[k].name);
        for (int k = 0; k < j; ++k)
            if (overlap(o, out.of[k])) return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, o.name, out.of[k].name);
    }
    return SFM_OK;
}

sfm_status check_workspace(const char* fn, const void* ws, int64_t have, int64_t need) {
    if (need <= 0) return SFM_OK;
    if (!ws || have < need)
        return fail(SFM_ERR_SHAPE, "%s: workspace of %lld bytes needed, %lld given", fn, (long long)need,
                    (long long)(ws ? have : 0));
    if (!aligned16(ws)) return fail(SFM_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    return SFM_OK;
}

sfm::RecParams params(const void* x, const void* r, const void* i, const float* lam, int64_t rows, int64_t L, int64_t tokens,
                      int64_t D, int64_t ldx, int64_t ldr, int64_t ldi, float c) {
    sfm::RecParams p{};
    p.x = x, p.r = r, p.i = i, p.lam = lam;
    p.ldx = ldx, p.ldr = ldr, p.ldi = ldi, p.tokens = tokens;
    p.rows = (int)rows, p.L = (int)L, p.D = (int)D, p.c = c;
    return p;
}

}  // namespace

extern "C" {

sfm_status sfm_gated_recurrence_fwd_ws_size(int64_t rows, int64_t L, int64_t tokens, int64_t D, int io_dtype,
                                            int64_t* bytes) {
    static const char* fn = "sfm_gated_recurrence_fwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, rows, L, tokens, true, D, io_dtype);
    if (st != SFM_OK) return st;
    const int64_t need = need_of_either(rows, L, tokens, D, io_dtype, false);
    if (need < 0) return too_large(fn, rows, tokens, D);
    *bytes = need;
    return ok();
}

sfm_status sfm_gated_recurrence_bwd_ws_size(int64_t rows, int64_t L, int64_t tokens, int64_t D, int io_dtype,
                                            int64_t* bytes) {
    static const char* fn = "sfm_gated_recurrence_bwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, rows, L, tokens, true, D, io_dtype);
    if (st != SFM_OK) return st;
    const int64_t need = need_of_either(rows, L, tokens, D, io_dtype, true);
    if (need < 0) return too_large(fn, rows, tokens, D);
    *bytes = need;
    return ok();
}

sfm_status sfm_gated_recurrence_fwd(const void* x, const void* r, const void* i, const float* lam, const float* h0, void* y,
                                    float* hT, const int32_t* offsets, int64_t rows, int64_t L, int64_t tokens, int64_t D,
                                    int64_t ldx, int64_t ldr, int64_t ldi, float c, int io_dtype, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_gated_recurrence_fwd";
    sfm_status st = check_sizes(fn, rows, L, tokens, offsets != nullptr, D, io_dtype);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, x, r, i, lam, tokens, D, ldx, ldr, ldi, sfm::rec_max_stride(L, io_bytes(io_dtype)), c, io_dtype);
    if (st != SFM_OK) return st;
    if (tokens > 0 && !y) return fail(SFM_ERR_NULL, "%s: y is required", fn);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(h0, 4) || !aligned_to(hT, 4) || !aligned_to(offsets, 4) || !aligned_to(y, e))
        return fail(SFM_ERR_ALIGN, "%s: h0, hT, offsets or y not aligned to its element", fn);
    const int64_t need = need_of(rows, L, tokens, D, offsets != nullptr, io_dtype, false);
    if (need < 0) return too_large(fn, rows, tokens, D);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SFM_OK) return st;
    Ranges in, out;
    in.add_inputs(x, r, i, lam, tokens, D, ldx, ldr, ldi, e);
    in.add("offsets", offsets, (rows + 1) * 4);
    in.add("h0", h0, rows * D * 4);
    out.add("y", y, tokens * D * e);
    out.add("hT", hT, rows * D * 4);
    out.add("workspace", workspace, need);
    st = check_ranges(fn, in, out);
    if (st != SFM_OK) return st;
    sfm::RecParams p = params(x, r, i, lam, rows, L, tokens, D, ldx, ldr, ldi, c);
    p.h0 = h0, p.y = y, p.hT = hT, p.offsets = offsets;
    take_plan(p, wide_tokens({x, r, i, y}, {ldx, ldr, ldi, D}, io_dtype), io_dtype, false, workspace);
    return hip_status(sfm::launch_rec_fwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

sfm_status sfm_gated_recurrence_bwd(const void* x, const void* r, const void* i, const float* lam, const float* h0,
                                    const void* y, const void* dy, const float* dhT, void* dx, void* dr, void* di,
                                    float* dlam, float* dh0, const int32_t* offsets, int64_t rows, int64_t L,
                                    int64_t tokens, int64_t D, int64_t ldx, int64_t ldr, int64_t ldi, float c, int io_dtype,
                                    void* workspace, int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_gated_recurrence_bwd";
    sfm_status st = check_sizes(fn, rows, L, tokens, offsets != nullptr, D, io_dtype);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, x, r, i, lam, tokens, D, ldx, ldr, ldi, sfm::rec_max_stride(L, io_bytes(io_dtype)), c, io_dtype);
    if (st != SFM_OK) return st;
    if (!dlam || (tokens > 0 && (!y || !dy || !dx || !dr || !di)))
        return fail(SFM_ERR_NULL, "%s: y, dy, dx, dr, di and dlam are required", fn);
    const int e = io_bytes(io_dtype);
    for (const void* t : {y, dy, (const void*)dx, (const void*)dr, (const void*)di})
        if (!aligned_to(t, e)) return fail(SFM_ERR_ALIGN, "%s: y, dy or a gradient not aligned to its element", fn);
    for (const void* t : {(const void*)h0, (const void*)dhT, (const void*)dh0, (const void*)dlam, (const void*)offsets})
        if (!aligned_to(t, 4)) return fail(SFM_ERR_ALIGN, "%s: h0, dhT, dh0, dlam or offsets not aligned to its element", fn);
    const int64_t need = need_of(rows, L, tokens, D, offsets != nullptr, io_dtype, true);
    if (need < 0) return too_large(fn, rows, tokens, D);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SFM_OK) return st;
    const int64_t nb = tokens * D * e, sb = rows * D * 4;
    Ranges in, out;
    in.add_inputs(x, r, i, lam, tokens, D, ldx, ldr, ldi, e);
    in.add("offsets", offsets, (rows + 1) * 4);
    in.add("h0", h0, sb);
    in.add("y", y, nb);
    in.add("dy", dy, nb);
    in.add("dhT", dhT, sb);
    out.add("dx", dx, nb);
    out.add("dr", dr, nb);
    out.add("di", di, nb);
    out.add("dlam", dlam, D * 4);
    out.add("dh0", dh0, sb);
    out.add("workspace", workspace, need);
    st = check_ranges(fn, in, out);
    if (st != SFM_OK) return st;
    sfm::RecParams p = params(x, r, i, lam, rows, L, tokens, D, ldx, ldr, ldi, c);
    p.h0 = h0, p.offsets = offsets, p.y = const_cast<void*>(y), p.dy = dy, p.dhT = dhT;
    p.dx = dx, p.dr = dr, p.di = di, p.dlam = dlam, p.dh0 = dh0;
    take_plan(p, wide_tokens({x, r, i, y, dy, dx, dr, di}, {ldx, ldr, ldi, D}, io_dtype), io_dtype, true, workspace);
    return hip_status(sfm::launch_rec_bwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

sfm_status sfm_gated_recurrence_step(const void* x, const void* r, const void* i, const float* lam, float* state,
                                     const int32_t* slots, void* y, int64_t rows, int64_t pool, int64_t D, int64_t ldx,
                                     int64_t ldr, int64_t ldi, float c, int io_dtype, void* stream) {
    static const char* fn = "sfm_gated_recurrence_step";
    sfm_status st = check_sizes(fn, rows, 1, rows, false, D, io_dtype);
    if (st != SFM_OK) return st;
    st = check_inputs(fn, x, r, i, lam, rows, D, ldx, ldr, ldi, 1LL << 36, c, io_dtype);
    if (st != SFM_OK) return st;
    if (!state || !y) return fail(SFM_ERR_NULL, "%s: state and y are required", fn);
    if (!sane(pool, 1 << 24)) return fail(SFM_ERR_SHAPE, "%s: a pool of %lld states", fn, (long long)pool);
    if (!slots && pool < rows)
        return fail(SFM_ERR_SHAPE, "%s: %lld states for %lld rows (no slots)", fn, (long long)pool, (long long)rows);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(state, 4) || !aligned_to(slots, 4) || !aligned_to(y, e))
        return fail(SFM_ERR_ALIGN, "%s: state, slots or y not aligned to its element", fn);
    Ranges in, out;
    in.add_inputs(x, r, i, lam, rows, D, ldx, ldr, ldi, e);
    in.add("slots", slots, rows * 4);
    out.add("state", state, pool * D * 4);
    out.add("y", y, rows * D * e);
    st = check_ranges(fn, in, out);
    if (st != SFM_OK) return st;
    sfm::RecParams p = params(x, r, i, lam, rows, 1, rows, D, ldx, ldr, ldi, c);
    p.hT = state, p.slots = slots, p.pool = pool, p.y = y;
    return hip_status(sfm::launch_rec_step(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
