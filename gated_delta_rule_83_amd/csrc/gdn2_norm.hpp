// gdn2_norm.hpp -- launch interface of the layer and root-mean-square norm
// (gdn2_operators_api.cpp to gdn2_norm.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

struct NormArgs {
  int64_t rows;
  int D;
  bool layer;  // false: root mean square
  bool bf16, wbf16;
  float eps;
  const void *x, *weight, *bias, *gate;
  void *y;
  const void *dy;
  void *dx, *dweight, *dbias, *dgate;
  void *workspace;
};

// Partial column sums of the weight's and the bias's gradient.
size_t norm_backward_workspace_bytes(int64_t rows, int D, bool bf16);
hipError_t launch_norm_forward(const NormArgs &p, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs &p, hipStream_t stream);

}  // namespace gdn2
