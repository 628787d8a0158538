// delta_bwd_bf16.hip -- the backward of the gated delta rule for bfloat16 tensors (delta_bwd.h).
#include "delta_bwd.h"

namespace sfm {

// Two bfloat16 parts to a computed operand; three on the way to the initial states' gradient, which is float32.
hipError_t launch_delta_bwd_bf16(const DeltaParams& p, hipStream_t s) {
    if (p.dh0) return p.dk <= 64 ? launch_backward<__bf16, 64, 3>(p, s) : launch_backward<__bf16, 128, 3>(p, s);
    return p.dk <= 64 ? launch_backward<__bf16, 64, 2>(p, s) : launch_backward<__bf16, 128, 2>(p, s);
}

}  // namespace sfm
