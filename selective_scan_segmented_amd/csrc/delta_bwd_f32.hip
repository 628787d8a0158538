// delta_bwd_f32.hip -- the backward of the gated delta rule for float32 tensors (delta_bwd.h).
#include "delta_bwd.h"

namespace sfm {

hipError_t launch_delta_bwd_f32(const DeltaParams& p, hipStream_t s) {
    return p.dk <= 64 ? launch_backward<float, 64, 1>(p, s) : launch_backward<float, 128, 1>(p, s);
}

}  // namespace sfm
