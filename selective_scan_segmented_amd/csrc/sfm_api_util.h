// sfm_api_util.h -- error reporting and argument checks shared by the C-ABI files.  Not part of the public ABI.
#pragma once

#include "sfm.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

namespace sfm {
namespace api {

extern thread_local std::string g_last_error;  // sfm_api.cpp; read by sfm_last_error()

inline sfm_status fail(sfm_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

inline sfm_status ok() {
    g_last_error.clear();
    return SFM_OK;
}

inline sfm_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(SFM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline int io_bytes(int io_dtype) { return io_dtype == SFM_F32 ? 4 : 2; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
    const char* name;
    uintptr_t lo, hi;
};

inline Range rng(const char* name, const void* p, int64_t bytes) {
    uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, lo + static_cast<uintptr_t>(bytes)};
}

inline bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

// products of positive sizes that must stay well inside int32 indexing of one
// (sample, channel) row and int64 element counts overall
inline bool sane(int64_t v, int64_t hi) { return v >= 1 && v <= hi; }

}  // namespace api
}  // namespace sfm
