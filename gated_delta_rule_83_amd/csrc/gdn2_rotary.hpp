// gdn2_rotary.hpp -- launch interface of the head norm and rotation by position
// (gdn2_attention_api.cpp to gdn2_rotary.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

struct RotaryArgs {
  int64_t tokens;
  int Hq, Hk, d, rot;
  bool norm, neighbours, bf16, wbf16;
  float eps;
  int64_t sq, sk;  // elements from a token to the next in q and k
  const void *q, *k, *qw, *kw;
  const int32_t *positions;
  const float *inv_freq;
  void *q_out, *k_out;
  // backward: the results' gradients (contiguous)
  const void *gq, *gk;
  void *dq, *dk, *dqw, *dkw;
  void *workspace;
};

constexpr int kRotaryMaxD = 1024;

size_t rotary_backward_workspace_bytes(int64_t tokens, int Hq, int Hk, int d);
hipError_t launch_rotary_forward(const RotaryArgs &p, hipStream_t stream);
hipError_t launch_rotary_backward(const RotaryArgs &p, hipStream_t stream);

}  // namespace gdn2
