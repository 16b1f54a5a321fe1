// gdn2_linattn_f32.hip -- sweep kernels of the linear attention with a decay for each head, fp32 inputs.

#include "gdn2_linattn_launch.h"

namespace gdn2 {

hipError_t launch_linattn_f32(const LinArgs& a, bool state, hipStream_t s) { return launch_lin_a<true>(a, state, s); }

}  // namespace gdn2
