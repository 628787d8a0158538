// delta_fwd_bf16.hip -- the chunked forward of the gated delta rule for bfloat16 tensors (delta_fwd.h, delta_narrow.h).
#include "delta_narrow.h"

namespace sfm {

// Computed operands have two bfloat16 parts where only bfloat16 outputs come of them (relative error 2^-17 against
// their rounding of 2^-9), three where the states are asked for, in float32.
hipError_t launch_delta_fwd_bf16(const DeltaParams& p, hipStream_t s) {
    if (p.hT) return p.dk <= 64 ? launch_forward<__bf16, 64, 3>(p, s) : launch_forward<__bf16, 128, 3>(p, s);
    return p.dk <= 64 ? launch_forward<__bf16, 64, 2>(p, s) : launch_forward<__bf16, 128, 2>(p, s);
}

}  // namespace sfm
