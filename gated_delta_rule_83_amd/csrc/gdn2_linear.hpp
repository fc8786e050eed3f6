// gdn2_linear.hpp -- launch interface of the gated linear recurrence
// (gdn2_operators_api.cpp to gdn2_linear.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

// Tokens a workgroup holds at once, and the spacing of the saved states.
constexpr int kLinTile = 64;
// Channels a workgroup owns.
constexpr int kLinChannels = 128;

struct LinearArgs {
  int B, T, D;
  int gates;  // gdn2_linear_gates
  bool bf16;
  const void *x, *a, *b;  // b unused in the tied forms
  const float *h0;
  // forward: outputs (o may be null: saved states only), last states, saved states
  void *o;
  float *h_T;
  float *ck;
  // backward: also ck as an input
  const void *dO;
  const float *dh_T;
  void *dx, *da, *db;
  float *dh0;
  const int32_t *cu;  // B + 1 offsets of packed sequences over T tokens, or null
  void *workspace;
};

// Saved states of a call: one row of D fp32 per kLinTile tokens of every
// sequence (packed: of the packed axis).
inline size_t linear_checkpoint_rows(int B, int T, bool packed) {
  const size_t tiles = ((size_t)T + kLinTile - 1) / kLinTile;
  return packed ? tiles : tiles * (size_t)B;
}

// Bytes of the words through which the tiles of a call are chained (a multiple of 16).
size_t linear_chain_bytes(int B, int T, int D, bool packed);

hipError_t launch_linear_forward(const LinearArgs &p, hipStream_t stream);
hipError_t launch_linear_backward(const LinearArgs &p, hipStream_t stream);
// One token: h_out = a h + b x, o = h_out, N = p.B rows of p.D (p.h0: h, p.h_T: h_out).
hipError_t launch_linear_step(const LinearArgs &p, hipStream_t stream);

}  // namespace gdn2
