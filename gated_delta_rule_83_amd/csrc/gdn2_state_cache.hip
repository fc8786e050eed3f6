// gdn2_state_cache.hip -- recurrent states written to a slot-indexed cache in
// 8 bits and read back.
//
// A row of d_v values shares one scale 2^e, the smallest power of two that
// keeps the row's largest magnitude within the format's largest value:
//   e4m3: 448 = 1.75 * 2^8,  int8: 127 = 1.984375 * 2^6.
// Dividing by a power of two is exact, so the only rounding is the one to the
// format's grid (half to even), and the stored byte is the scale's fp32
// exponent field e + 127: the factor 2^-e or 2^e is assembled from it with a
// shift. Both passes are bound by HBM: 5 bytes a value and 1 a row. The fp32
// side is read or written once, nontemporal: 256 states of 16 x 128 x 128 are
// stored in 57 us and loaded in 49 (5.9 and 6.8 TB/s; 66 and 67 us without,
// two rows of a thread in flight against 59 and 49 us with four).
#include "gdn2_device.hpp"
#include "gdn2_state_cache.hpp"

#include "gdn2.h"

namespace gdn2 {

namespace {

constexpr int kNT = 256;
constexpr int kUnroll = 2;  // rows of a thread in flight

// Rows are taken by TPR = d_v / 8 lanes: 4 values of the row's first half and
// 4 of its second each, so that both 16-byte loads of a row are contiguous.
template <int DV> struct Rows {
  static constexpr int TPR = DV / 8, PER = kNT / TPR, BLOCK = PER * kUnroll;  // rows a pass, rows a workgroup
};

template <int FMT> __device__ __forceinline__ uint32_t scale_byte(uint32_t big) {
  // big: bits of the largest magnitude; inf or NaN give 255
  constexpr uint32_t top = FMT == GDN2_CACHE_E4M3 ? 0x600000u : 0x7e0000u;
  constexpr int bits = FMT == GDN2_CACHE_E4M3 ? 8 : 6;
  if (big >= 0x7f800000u) return 255u;
  const int e = (int)(big >> 23) - bits + ((big & 0x7fffffu) > top ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e);
}

// Largest code a row may use: the format's own, but for rows from the last
// binade whose largest value could round up to 2^128, which fp32 cannot hold.
template <int FMT> __device__ __forceinline__ float largest_code(uint32_t sb) {
  if constexpr (FMT == GDN2_CACHE_E4M3) return sb == 254u - 8 + 1 ? 240.f : 448.f;
  return sb == 254u - 6 + 1 ? 63.f : 127.f;
}

// Four values to four codes.
template <int FMT> __device__ __forceinline__ uint32_t encode(floatx4 v) {
  if constexpr (FMT == GDN2_CACHE_E4M3) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
  } else {
    uint32_t r = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) r |= ((uint32_t)(int)__builtin_rintf(v[c]) & 255u) << (8 * c);
    return r;
  }
}

template <int FMT> __device__ __forceinline__ floatx4 decode(uint32_t r) {
  if constexpr (FMT == GDN2_CACHE_E4M3) {
    const floatx2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)r, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)r, true);
    return floatx4{lo[0], lo[1], hi[0], hi[1]};
  } else {
    return floatx4{(float)(int8_t)r, (float)(int8_t)(r >> 8), (float)(int8_t)(r >> 16), (float)((int32_t)r >> 24)};
  }
}

template <int FMT, int DV>
__global__ __launch_bounds__(kNT) void store_kernel(StateCacheArgs p, int per_entry) {
  using R = Rows<DV>;
  const int n = blockIdx.x / per_entry, blk = blockIdx.x - n * per_entry;
  const int tid = threadIdx.x, l = tid % R::TPR;
  const int slot = p.slots[n];
  if (slot < 0 || slot >= p.P) return;
  floatx4 v[kUnroll][2];
  int row[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    row[i] = blk * R::BLOCK + i * R::PER + tid / R::TPR;
    const int r = row[i] < p.rows ? row[i] : p.rows - 1;
    const float *s = p.S + ((size_t)n * p.rows + r) * DV;
    v[i][0] = __builtin_nontemporal_load(reinterpret_cast<const floatx4 *>(s + 4 * l));
    v[i][1] = __builtin_nontemporal_load(reinterpret_cast<const floatx4 *>(s + DV / 2 + 4 * l));
  }
  // a slot named twice keeps its last entry
  int later = 0;
  for (int j = n + 1 + tid; j < p.N; j += kNT) later |= p.slots[j] == slot;
  if (__syncthreads_or(later)) return;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    uint32_t big = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t m = __float_as_uint(v[i][c >> 2][c & 3]) & 0x7fffffffu;
      big = m > big ? m : big;
    }
#pragma unroll
    for (int off = 1; off < R::TPR; off <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)big, off, 64);
      big = o > big ? o : big;
    }
    const uint32_t sb = scale_byte<FMT>(big);
    if (row[i] >= p.rows) continue;
    const float inv = sb == 255u ? 0.f : __uint_as_float((254u - sb) << 23);
    const float lim = largest_code<FMT>(sb);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[i][c >> 2][c & 3] = __builtin_amdgcn_fmed3f(v[i][c >> 2][c & 3] * inv, -lim, lim);
    const size_t at = (size_t)slot * p.rows + row[i];
    uint32_t *c = reinterpret_cast<uint32_t *>(p.cache + at * DV);
    c[l] = encode<FMT>(v[i][0]);
    c[DV / 8 + l] = encode<FMT>(v[i][1]);
    if (l == 0) p.scales[at] = (uint8_t)sb;
  }
}

template <int FMT, int DV>
__global__ __launch_bounds__(kNT) void load_kernel(StateCacheArgs p, int per_entry) {
  using R = Rows<DV>;
  const int n = blockIdx.x / per_entry, blk = blockIdx.x - n * per_entry;
  const int tid = threadIdx.x, l = tid % R::TPR;
  const int slot = p.slots[n];
  const bool in = slot >= 0 && slot < p.P;
  uint32_t c[kUnroll][2], sb[kUnroll];
  int row[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    row[i] = blk * R::BLOCK + i * R::PER + tid / R::TPR;
    c[i][0] = c[i][1] = sb[i] = 0;
    if (in) {
      const size_t at = (size_t)slot * p.rows + (row[i] < p.rows ? row[i] : p.rows - 1);
      const uint32_t *q = reinterpret_cast<const uint32_t *>(p.cache + at * DV);
      c[i][0] = q[l];
      c[i][1] = q[DV / 8 + l];
      sb[i] = p.scales[at];
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    if (row[i] >= p.rows) continue;
    const float f = sb[i] == 255u ? __builtin_nanf("") : __uint_as_float(sb[i] << 23);
    float *s = p.S + ((size_t)n * p.rows + row[i]) * DV;
    __builtin_nontemporal_store(decode<FMT>(c[i][0]) * f, reinterpret_cast<floatx4 *>(s + 4 * l));
    __builtin_nontemporal_store(decode<FMT>(c[i][1]) * f, reinterpret_cast<floatx4 *>(s + DV / 2 + 4 * l));
  }
}

template <int FMT, int DV> hipError_t launch(const StateCacheArgs &p, bool store, hipStream_t st) {
  const int per = (int)state_cache_groups(p.rows, DV);
  static_assert(Rows<DV>::BLOCK == 2 * 256 / (DV / 8), "state_cache_groups");
  const dim3 grid((unsigned)((size_t)p.N * per));
  if (store)
    hipLaunchKernelGGL((store_kernel<FMT, DV>), grid, dim3(kNT), 0, st, p, per);
  else
    hipLaunchKernelGGL((load_kernel<FMT, DV>), grid, dim3(kNT), 0, st, p, per);
  return hipGetLastError();
}

template <int FMT> hipError_t launch_dv(const StateCacheArgs &p, bool store, hipStream_t st) {
  switch (p.d_v) {
    case 16: return launch<FMT, 16>(p, store, st);
    case 32: return launch<FMT, 32>(p, store, st);
    case 64: return launch<FMT, 64>(p, store, st);
    case 128: return launch<FMT, 128>(p, store, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_any(const StateCacheArgs &p, bool store, hipStream_t st) {
  return p.format == GDN2_CACHE_E4M3 ? launch_dv<GDN2_CACHE_E4M3>(p, store, st)
                                     : launch_dv<GDN2_CACHE_INT8>(p, store, st);
}

}  // namespace

hipError_t launch_state_cache_store(const StateCacheArgs &p, hipStream_t st) { return launch_any(p, true, st); }
hipError_t launch_state_cache_load(const StateCacheArgs &p, hipStream_t st) { return launch_any(p, false, st); }

}  // namespace gdn2
