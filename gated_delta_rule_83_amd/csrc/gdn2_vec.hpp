// gdn2_vec.hpp -- wide loads and stores of N consecutive values of a tensor,
// and sums over groups of lanes (gfx950 only).
#pragma once

#include "gdn2_device.hpp"

namespace gdn2 {

typedef uint32_t uintx2 __attribute__((ext_vector_type(2)));
typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));

// N values as they lie in memory.
template <bool BF16, int N> struct Raw;
template <> struct Raw<false, 4> {
  floatx4 v;
  __device__ __forceinline__ float operator[](int c) const { return v[c]; }
};
template <> struct Raw<true, 8> {
  uintx4 v;
  __device__ __forceinline__ float operator[](int c) const {
    return __uint_as_float(c & 1 ? v[c >> 1] & 0xffff0000u : v[c >> 1] << 16);
  }
};
template <> struct Raw<true, 4> {
  uintx2 v;
  __device__ __forceinline__ float operator[](int c) const {
    return __uint_as_float(c & 1 ? v[c >> 1] & 0xffff0000u : v[c >> 1] << 16);
  }
};
template <> struct Raw<false, 1> {
  float v;
  __device__ __forceinline__ float operator[](int) const { return v; }
};
template <> struct Raw<true, 1> {
  uint16_t v;
  __device__ __forceinline__ float operator[](int) const { return bf16_to_f32(v); }
};

// A wave-uniform base and a 32-bit lane offset (bytes): the row's part of an
// address costs no vector instruction. Nontemporal: for what is read once.
template <bool BF16, int N> __device__ __forceinline__ Raw<BF16, N> load_raw(const char *base, uint32_t off) {
  using V = decltype(Raw<BF16, N>::v);
  return Raw<BF16, N>{__builtin_nontemporal_load(reinterpret_cast<const V *>(base + off))};
}

template <bool BF16, int N> __device__ __forceinline__ void load_f(float (&f)[N], const void *p, size_t i) {
  using T = typename Elem<BF16>::T;
  const Raw<BF16, N> r{*reinterpret_cast<const decltype(Raw<BF16, N>::v) *>(static_cast<const T *>(p) + i)};
#pragma unroll
  for (int c = 0; c < N; ++c) f[c] = r[c];
}

template <bool BF16, int N> __device__ __forceinline__ void store_at(char *p, const float (&f)[N]) {
  using T = typename Elem<BF16>::T;
  struct { T e[N]; } v;
#pragma unroll
  for (int c = 0; c < N; ++c) Elem<BF16>::st(&v.e[c], f[c]);
  __builtin_memcpy(__builtin_assume_aligned(p, sizeof(T) * N < 16 ? sizeof(T) * N : 16), &v, sizeof(v));
}
template <bool BF16, int N> __device__ __forceinline__ void store_f(void *p, size_t i, const float (&f)[N]) {
  store_at<BF16>(static_cast<char *>(p) + i * sizeof(typename Elem<BF16>::T), f);
}

// x of the lane that DPP control CTRL pairs with this one. The empty asm keeps
// shifts of several values apart (see row_shr).
template <int CTRL> __device__ __forceinline__ float dpp_pair(float x) {
  asm volatile("" : "+v"(x));
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over each group of N consecutive lanes (a power of two up to 64), the
// same value and rounding in all of them.
template <int N> __device__ __forceinline__ float lane_sum(float x) {
  if constexpr (N >= 2) x += dpp_pair<0xb1>(x);   // quad_perm [1, 0, 3, 2]
  if constexpr (N >= 4) x += dpp_pair<0x4e>(x);   // quad_perm [2, 3, 0, 1]
  if constexpr (N >= 8) x += dpp_pair<0x141>(x);  // row_half_mirror: the other quad of 8
  if constexpr (N >= 16) x += dpp_pair<0x140>(x);  // row_mirror: the other 8 of 16
  if constexpr (N >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (N >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

}  // namespace gdn2
