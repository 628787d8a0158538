// sfm_rope_api.cpp -- the C ABI of the norm and rotation of queries and keys (declared in include/sfm.h): checks and dispatch.
#include "sfm.h"

#include <hip/hip_runtime.h>

#include <initializer_list>

#include "sfm_api_util.h"
#include "sfm_rope.h"

using namespace sfm::api;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sfm_status check_sizes(const char* fn, int64_t tokens, int64_t Hq, int64_t Hk, int64_t d, int io_dtype) {
    if (io_dtype != SFM_F32 && io_dtype != SFM_BF16) return fail(SFM_ERR_DTYPE, "%s: io_dtype %d", fn, io_dtype);
    if (tokens < 0 || tokens > (1LL << 31) - 1 || !sane(Hq, 4096) || !sane(Hk, 4096) || !sane(d, sfm::kRopeMaxD))
        return fail(SFM_ERR_SHAPE, "%s: tokens=%lld, %lld and %lld heads of %lld (1 to %d) out of range", fn,
                    (long long)tokens, (long long)Hq, (long long)Hk, (long long)d, sfm::kRopeMaxD);
    return SFM_OK;
}

// The checks that both directions share; fills the call's sizes.
sfm_status fill(const char* fn, sfm::RopeParams& p, const void* q, const void* k, const float* wq, const float* wk,
                const int32_t* positions, const float* freqs, int64_t tokens, int64_t period, int64_t Hq, int64_t Hk,
                int64_t d, int64_t rot, int64_t axes, const int64_t* sections, int64_t ldq, int64_t ldk, float eps,
                int io_dtype, int flags) {
    const sfm_status st = check_sizes(fn, tokens, Hq, Hk, d, io_dtype);
    if (st != SFM_OK) return st;
    if (flags & ~(SFM_QK_NORM | SFM_QK_NEIGHBOURS)) return fail(SFM_ERR_SHAPE, "%s: unknown flags 0x%x", fn, flags);
    if (rot < 0 || rot > d || rot % 2) return fail(SFM_ERR_SHAPE, "%s: rot=%lld of heads of %lld", fn, (long long)rot, (long long)d);
    if (tokens > 0 && (!q || !k)) return fail(SFM_ERR_NULL, "%s: q and k are required", fn);
    if (rot > 0 && (!freqs || (tokens > 0 && !positions)))
        return fail(SFM_ERR_NULL, "%s: positions and freqs are required with a rotation", fn);
    if (ldq < Hq * d || ldk < Hk * d || ldq > 1 << 29 || ldk > 1 << 29)
        return fail(SFM_ERR_SHAPE, "%s: token strides %lld, %lld below the heads' widths (or too large)", fn,
                    (long long)ldq, (long long)ldk);
    if (!(flags & SFM_QK_NORM) && (wq || wk)) return fail(SFM_ERR_SHAPE, "%s: weights without the norm", fn);
    // (a normal float32: squares too small for one then vanish beside it)
    if ((flags & SFM_QK_NORM) && !(eps >= 1.17549435e-38f && eps <= 1e30f)) return fail(SFM_ERR_SHAPE, "%s: eps=%g", fn, (double)eps);
    if (rot > 0) {
        if (!sane(axes, sfm::kRopeMaxAxes)) return fail(SFM_ERR_SHAPE, "%s: %lld position axes", fn, (long long)axes);
        if (tokens > 0 && (period < 1 || tokens % period))
            return fail(SFM_ERR_SHAPE, "%s: %lld tokens are not whole runs of %lld positions", fn, (long long)tokens, (long long)period);
        int64_t end = 0;
        for (int a = 0; a < axes; ++a) {
            const int64_t n = sections ? sections[a] : axes == 1 ? rot / 2 : -1;
            if (n < 0 || n > rot / 2) return fail(SFM_ERR_SHAPE, "%s: sections of the position axes are required", fn);
            p.ends[a] = (int)(end += n);
        }
        if (end != rot / 2)
            return fail(SFM_ERR_SHAPE, "%s: sections of %lld pairs in place of %lld", fn, (long long)end, (long long)(rot / 2));
    }
    const uintptr_t e = io_bytes(io_dtype);
    if (!aligned_to(q, e) || !aligned_to(k, e)) return fail(SFM_ERR_ALIGN, "%s: q or k not aligned to its element", fn);
    for (const void* t : {(const void*)wq, (const void*)wk, (const void*)positions, (const void*)freqs})
        if (!aligned_to(t, 4)) return fail(SFM_ERR_ALIGN, "%s: weights, positions or freqs not aligned to the element", fn);
    p.side[0].x = q, p.side[0].w = wq, p.side[0].ld = ldq, p.side[0].heads = (int)Hq;
    p.side[1].x = k, p.side[1].w = wk, p.side[1].ld = ldk, p.side[1].heads = (int)Hk;
    p.positions = positions, p.freqs = freqs, p.tokens = tokens, p.period = period < 1 ? 1 : period;
    p.d = (int)d, p.rot = (int)rot, p.axes = rot > 0 ? (int)axes : 1, p.eps = eps;
    p.norm = flags & SFM_QK_NORM ? 1 : 0, p.neighbours = flags & SFM_QK_NEIGHBOURS ? 1 : 0;
    return SFM_OK;
}

// Bytes that all addresses are a multiple of, at most 16.
int alignment(std::initializer_list<const void*> tensors) {
    uintptr_t all = 16;
    for (const void* t : tensors) all |= reinterpret_cast<uintptr_t>(t);
    return (int)(all & -all);
}

struct Ranges {
    Range of[8];
    int n = 0;
    void add(const char* name, const void* p, int64_t bytes) {
        if (p && bytes > 0) of[n++] = rng(name, p, bytes);
    }
    void add_inputs(const sfm::RopeParams& p, int e) {
        if (p.tokens > 0)
            for (int s = 0; s < 2; ++s)
                add(s ? "k" : "q", p.side[s].x, ((p.tokens - 1) * p.side[s].ld + (int64_t)p.side[s].heads * p.d) * e);
        add("wq", p.side[0].w, p.d * 4);
        add("wk", p.side[1].w, p.d * 4);
        if (p.rot > 0) {
            if (p.tokens > 0) add("positions", p.positions, p.period * p.axes * 4);
            add("freqs", p.freqs, p.rot * 2);
        }
    }
};

sfm_status check_ranges(const char* fn, const Ranges& in, const Ranges& out) {
    for (int j = 0; j < out.n; ++j) {
        for (int k = 0; k < in.n; ++k)
            if (overlap(out.of[j], in.of[k])) return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, out.of[j].name, in.of[k].name);
        for (int k = 0; k < j; ++k)
            if (overlap(out.of[j], out.of[k])) return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, out.of[j].name, out.of[k].name);
    }
    return SFM_OK;
}

}  // namespace

extern "C" {

sfm_status sfm_qk_norm_rope_fwd(const void* q, const void* k, const float* wq, const float* wk, const int32_t* positions,
                                const float* freqs, void* qo, void* ko, int64_t tokens, int64_t period, int64_t Hq,
                                int64_t Hk, int64_t d, int64_t rot, int64_t axes, const int64_t* sections, int64_t ldq,
                                int64_t ldk, float eps, int io_dtype, int flags, void* stream) {
    static const char* fn = "sfm_qk_norm_rope_fwd";
    sfm::RopeParams p{};
    sfm_status st = fill(fn, p, q, k, wq, wk, positions, freqs, tokens, period, Hq, Hk, d, rot, axes, sections, ldq, ldk,
                         eps, io_dtype, flags);
    if (st != SFM_OK) return st;
    if (tokens == 0) return ok();
    if (!qo || !ko) return fail(SFM_ERR_NULL, "%s: qo and ko are required", fn);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(qo, e) || !aligned_to(ko, e)) return fail(SFM_ERR_ALIGN, "%s: qo or ko not aligned to its element", fn);
    Ranges in, out;
    in.add_inputs(p, e);
    out.add("qo", qo, tokens * Hq * d * e);
    out.add("ko", ko, tokens * Hk * d * e);
    st = check_ranges(fn, in, out);
    if (st != SFM_OK) return st;
    p.side[0].y = qo, p.side[1].y = ko;
    sfm::plan_rope(p, e, alignment({q, k, qo, ko}), false);
    return hip_status(sfm::launch_rope_fwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

sfm_status sfm_qk_norm_rope_bwd_ws_size(int64_t tokens, int64_t Hq, int64_t Hk, int64_t d, int want_weights, int io_dtype,
                                        int64_t* bytes) {
    static const char* fn = "sfm_qk_norm_rope_bwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, tokens, Hq, Hk, d, io_dtype);
    if (st != SFM_OK) return st;
    *bytes = want_weights ? 2 * (int64_t)sfm::kRopeParts * d * 4 : 0;
    return ok();
}

sfm_status sfm_qk_norm_rope_bwd(const void* dqo, const void* dko, const void* q, const void* k, const float* wq,
                                const float* wk, const int32_t* positions, const float* freqs, void* dq, void* dk, float* dwq,
                                float* dwk, int64_t tokens, int64_t period, int64_t Hq, int64_t Hk, int64_t d, int64_t rot,
                                int64_t axes, const int64_t* sections, int64_t ldq, int64_t ldk, float eps, int io_dtype,
                                int flags, void* workspace, int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_qk_norm_rope_bwd";
    sfm::RopeParams p{};
    sfm_status st = fill(fn, p, q, k, wq, wk, positions, freqs, tokens, period, Hq, Hk, d, rot, axes, sections, ldq, ldk,
                         eps, io_dtype, flags);
    if (st != SFM_OK) return st;
    if (tokens > 0 && (!dqo || !dko || !dq || !dk)) return fail(SFM_ERR_NULL, "%s: dqo, dko, dq and dk are required", fn);
    if (!p.norm && (dwq || dwk)) return fail(SFM_ERR_SHAPE, "%s: gradients of weights without the norm", fn);
    const int e = io_bytes(io_dtype);
    for (const void* t : {dqo, dko, (const void*)dq, (const void*)dk})
        if (!aligned_to(t, e)) return fail(SFM_ERR_ALIGN, "%s: a gradient is not aligned to its element", fn);
    if (!aligned_to(dwq, 4) || !aligned_to(dwk, 4)) return fail(SFM_ERR_ALIGN, "%s: dwq or dwk not aligned to its element", fn);
    const int64_t need = dwq || dwk ? 2 * (int64_t)sfm::kRopeParts * d * 4 : 0;
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(SFM_ERR_SHAPE, "%s: workspace of %lld bytes needed, %lld given", fn, (long long)need,
                    (long long)(workspace ? workspace_bytes : 0));
    if (need > 0 && !aligned16(workspace)) return fail(SFM_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    const int64_t nq = tokens * Hq * d * e, nk = tokens * Hk * d * e;
    Ranges in, out;
    in.add_inputs(p, e);
    in.add("dqo", dqo, nq);
    in.add("dko", dko, nk);
    out.add("dq", dq, nq);
    out.add("dk", dk, nk);
    out.add("dwq", dwq, d * 4);
    out.add("dwk", dwk, d * 4);
    out.add("workspace", need > 0 ? workspace : nullptr, need);
    st = check_ranges(fn, in, out);
    if (st != SFM_OK) return st;
    if (tokens == 0 && !dwq && !dwk) return ok();
    p.side[0].dy = dqo, p.side[1].dy = dko, p.side[0].y = dq, p.side[1].y = dk, p.side[0].dw = dwq, p.side[1].dw = dwk;
    p.part = need > 0 ? static_cast<float*>(workspace) : nullptr;
    sfm::plan_rope(p, e, alignment({q, k, dqo, dko, dq, dk}), true);
    return hip_status(sfm::launch_rope_bwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
