// sfm_norm_api.cpp -- the C ABI of the channel-last group norm (declared in include/sfm.h): checks and dispatch.
#include "sfm.h"

#include <hip/hip_runtime.h>

#include "sfm_api_util.h"
#include "sfm_norm.h"

using namespace sfm::api;

namespace {

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sfm_status check_sizes(const char* fn, int64_t N, int64_t L, int64_t C, int64_t G, int act, int io_dtype) {
    if (io_dtype != SFM_F32 && io_dtype != SFM_BF16) return fail(SFM_ERR_DTYPE, "%s: io_dtype %d", fn, io_dtype);
    if (!sane(N, 1 << 24) || !sane(L, 1 << 24) || !sane(C, 1 << 16) || !sane(G, C) || C % G)
        return fail(SFM_ERR_SHAPE, "%s: N=%lld L=%lld C=%lld G=%lld (out of range, or G does not divide C)", fn,
                    (long long)N, (long long)L, (long long)C, (long long)G);
    if (N * L > (1LL << 40) / C || N * C >= (1LL << 31)) return fail(SFM_ERR_SHAPE, "%s: tensor too large", fn);
    if (act != SFM_ACT_NONE && act != SFM_ACT_SILU) return fail(SFM_ERR_SHAPE, "%s: act=%d", fn, act);
    return SFM_OK;
}

// The plan depends on the alignment of the tensors only through `aligned`; the workspace is sized for either.
int64_t workspace_need(sfm::NormParams p, int e, bool bwd) {
    const int64_t a = sfm::plan_norm(p, e, true, bwd), b = sfm::plan_norm(p, e, false, bwd);
    return a > b ? a : b;
}

sfm::NormParams sizes(int64_t N, int64_t L, int64_t C, int64_t G, int act) {
    sfm::NormParams p{};
    p.N = N, p.L = L, p.C = (int)C, p.G = (int)G, p.act = act;
    return p;
}

sfm_status check_workspace(const char* fn, const void* ws, int64_t have, int64_t need) {
    if (need <= 0) return SFM_OK;
    if (!ws || have < need)
        return fail(SFM_ERR_SHAPE, "%s: workspace of %lld bytes needed, %lld given", fn, (long long)need,
                    (long long)(ws ? have : 0));
    if (!aligned16(ws)) return fail(SFM_ERR_ALIGN, "%s: workspace not 16-byte aligned", fn);
    return SFM_OK;
}

sfm_status check_ranges(const char* fn, const Range* ins, int ni, const Range* outs, int no) {
    for (int i = 0; i < no; ++i) {
        if (outs[i].lo == 0) continue;
        for (int j = 0; j < ni; ++j)
            if (ins[j].lo != 0 && overlap(outs[i], ins[j]))
                return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[i].name, ins[j].name);
        for (int j = 0; j < i; ++j)
            if (outs[j].lo != 0 && overlap(outs[i], outs[j]))
                return fail(SFM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[i].name, outs[j].name);
    }
    return SFM_OK;
}

}  // namespace

extern "C" {

sfm_status sfm_group_norm_fwd_ws_size(int64_t N, int64_t L, int64_t C, int64_t G, int io_dtype, int64_t* bytes) {
    static const char* fn = "sfm_group_norm_fwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, N, L, C, G, 0, io_dtype);
    if (st != SFM_OK) return st;
    *bytes = workspace_need(sizes(N, L, C, G, 0), io_bytes(io_dtype), false);
    return ok();
}

sfm_status sfm_group_norm_bwd_ws_size(int64_t N, int64_t L, int64_t C, int64_t G, int want_weights, int io_dtype,
                                      int64_t* bytes) {
    static const char* fn = "sfm_group_norm_bwd_ws_size";
    if (!bytes) return fail(SFM_ERR_NULL, "%s: bytes is required", fn);
    const sfm_status st = check_sizes(fn, N, L, C, G, 0, io_dtype);
    if (st != SFM_OK) return st;
    sfm::NormParams p = sizes(N, L, C, G, 0);
    float any = 0.0f;
    p.dw = want_weights ? &any : nullptr;  // plan_norm only asks whether it is there
    *bytes = workspace_need(p, io_bytes(io_dtype), true);
    return ok();
}

sfm_status sfm_group_norm_fwd(const void* x, const float* w, const float* b, void* y, float* mean, float* rstd,
                              int64_t N, int64_t L, int64_t C, int64_t G, float eps, int act, int io_dtype,
                              void* workspace, int64_t workspace_bytes, void* stream) {
    static const char* fn = "sfm_group_norm_fwd";
    if (!x || !y || !mean || !rstd) return fail(SFM_ERR_NULL, "%s: x, y, mean and rstd are required", fn);
    sfm_status st = check_sizes(fn, N, L, C, G, act, io_dtype);
    if (st != SFM_OK) return st;
    if (!(eps >= 0.0f)) return fail(SFM_ERR_SHAPE, "%s: eps=%g", fn, (double)eps);
    const int e = io_bytes(io_dtype);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(w, 4) || !aligned_to(b, 4) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return fail(SFM_ERR_ALIGN, "%s: a tensor is not aligned to its element", fn);
    sfm::NormParams p = sizes(N, L, C, G, act);
    const int64_t need = workspace_need(p, e, false);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SFM_OK) return st;
    const int64_t nb = N * L * C * e;
    const Range ins[] = {rng("x", x, nb), rng("w", w, w ? C * 4 : 0), rng("b", b, b ? C * 4 : 0)};
    const Range outs[] = {rng("y", y, nb), rng("mean", mean, N * G * 4), rng("rstd", rstd, N * G * 4),
                          rng("workspace", need ? workspace : nullptr, need)};
    st = check_ranges(fn, ins, 3, outs, 4);
    if (st != SFM_OK) return st;
    p.x = x, p.w = w, p.b = b, p.y = y, p.mean = mean, p.rstd = rstd, p.eps = eps;
    p.part = static_cast<float*>(workspace);
    sfm::plan_norm(p, e, aligned16(x) && aligned16(y), false);
    return hip_status(sfm::launch_group_norm_fwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

sfm_status sfm_group_norm_bwd(const void* dy, const void* x, const float* mean, const float* rstd, const float* w,
                              const float* b, void* dx, float* dw, float* db, int64_t N, int64_t L, int64_t C,
                              int64_t G, int act, int io_dtype, void* workspace, int64_t workspace_bytes,
                              void* stream) {
    static const char* fn = "sfm_group_norm_bwd";
    if (!dy || !x || !mean || !rstd || !dx) return fail(SFM_ERR_NULL, "%s: dy, x, mean, rstd and dx are required", fn);
    sfm_status st = check_sizes(fn, N, L, C, G, act, io_dtype);
    if (st != SFM_OK) return st;
    const int e = io_bytes(io_dtype);
    if (!aligned_to(dy, e) || !aligned_to(x, e) || !aligned_to(dx, e) || !aligned_to(w, 4) || !aligned_to(b, 4) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dw, 4) || !aligned_to(db, 4))
        return fail(SFM_ERR_ALIGN, "%s: a tensor is not aligned to its element", fn);
    sfm::NormParams p = sizes(N, L, C, G, act);
    p.dw = dw, p.db = db;
    const int64_t need = workspace_need(p, e, true);
    st = check_workspace(fn, workspace, workspace_bytes, need);
    if (st != SFM_OK) return st;
    const int64_t nb = N * L * C * e, cb = C * 4, sb = N * G * 4;
    const Range ins[] = {rng("dy", dy, nb),   rng("x", x, nb),           rng("mean", mean, sb),
                         rng("rstd", rstd, sb), rng("w", w, w ? cb : 0), rng("b", b, b ? cb : 0)};
    const Range outs[] = {rng("dx", dx, nb), rng("dw", dw, dw ? cb : 0), rng("db", db, db ? cb : 0),
                          rng("workspace", need ? workspace : nullptr, need)};
    st = check_ranges(fn, ins, 6, outs, 4);
    if (st != SFM_OK) return st;
    p.dy = dy, p.x = x, p.w = w, p.b = b, p.y = dx;
    p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
    p.part = need > 0 ? static_cast<float*>(workspace) : nullptr;
    sfm::plan_norm(p, e, aligned16(dy) && aligned16(x) && aligned16(dx), true);
    return hip_status(sfm::launch_group_norm_bwd(p, io_dtype, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
