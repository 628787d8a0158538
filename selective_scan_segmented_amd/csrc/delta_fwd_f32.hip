// delta_fwd_f32.hip -- the chunked forward of the gated delta rule for float32 tensors (delta_fwd.h, delta_narrow.h).
#include "delta_narrow.h"

namespace sfm {

hipError_t launch_delta_fwd_f32(const DeltaParams& p, hipStream_t s) {
    return p.dk <= 64 ? launch_forward<float, 64, 1>(p, s) : launch_forward<float, 128, 1>(p, s);
}

}  // namespace sfm
