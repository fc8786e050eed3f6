// gdn2_state_cache.hpp -- launch interface of the 8-bit state cache
// (gdn2_operators_api.cpp to gdn2_state_cache.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

struct StateCacheArgs {
  int N, P, rows, d_v;  // entries, slots, rows of a state, values of a row
  int format;           // gdn2_cache_format
  float *S;             // read by the store, written by the load
  const int32_t *slots;
  uint8_t *cache, *scales;
};

// Workgroups of one state: 256 threads take 8 values each of two rows.
inline size_t state_cache_groups(int rows, int d_v) {
  const size_t per = 2 * 256 / (d_v / 8);
  return ((size_t)rows + per - 1) / per;
}

hipError_t launch_state_cache_store(const StateCacheArgs &p, hipStream_t stream);
hipError_t launch_state_cache_load(const StateCacheArgs &p, hipStream_t stream);

}  // namespace gdn2
