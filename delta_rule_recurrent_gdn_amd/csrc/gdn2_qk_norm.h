// gdn2_qk_norm.h -- argument block and launchers of the q/k head norms with rotation. Not a public header.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

struct QkNormSide {              // q or k
  const void* x;                 // [tokens] rows of heads x D, x_stride elements apart
  const void* dy;                // backward: gradient of y, contiguous rows
  void* y;                       // forward: y; backward: dx; rows y_stride elements apart
  const float* w;                // [D], nullable (ones)
  float* dw;                     // [D], nullable
  int heads;
  int64_t x_stride, y_stride;
  float scale;                   // of y
};

struct QkNormArgs {
  QkNormSide s[2];               // q, k
  const int64_t* pos;            // positions[n % period], null: n % period
  const float* inv_freq;         // [rot / 2]
  int64_t tokens, period;
  int D, rot;
  float eps, inv_count;          // 1 / D, or 1 for the L2 norm
  bool interleaved, f32, f32_dy;
  float* partial;                // backward: [workgroups][2][D]
};

hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s);
hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s);
// workgroups of the backward, each with 2 D partial sums of the weights' gradients
int qk_norm_bwd_workgroups(int64_t tokens, int Hq, int Hk, int D);

}  // namespace gdn2
