// gdn2_linattn_bf16.hip -- sweep kernels of the linear attention with a decay for each head, bf16 inputs.

#include "gdn2_linattn_launch.h"

namespace gdn2 {

hipError_t launch_linattn_bf16(const LinArgs& a, bool state, hipStream_t s) { return launch_lin_a<false>(a, state, s); }

}  // namespace gdn2
