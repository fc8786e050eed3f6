// gdn2_attention_decode.hip -- attention of one new token a sequence over a
// paged key-value cache, and that cache's writes.
//
// The cache is read once, which bounds the call: 2 d values a key and key head,
// of which 16 query heads' products cost the matrix cores little. A workgroup
// takes a span of one sequence's keys and one key head, a wave every fourth tile
// of 32 keys, straight from memory to registers, the next tile's loads out before
// this one's are used (N4 131072 tokens: 111 us without, 88 with, 86 as it stands: 6.9 TB/s and the join):
//  - scores transposed (keys as rows), 16 x 16: a key's row is an A operand as it
//    lies, 8 values a lane;
//  - o transposed, too: row m of block r is channel m D / 16 + r, so a lane's
//    piece of D / 16 neighbouring channels serves D / 16 blocks, and the pairs of
//    keys that an operand's words hold come from two loads by one byte permute.
// Softmax state is a wave's own, joined over the waves in LDS and over the spans
// by a second kernel.
#include "gdn2_attention_device.hpp"

namespace gdn2 {
namespace {

using namespace attn;

constexpr int kTileKeys = 32, kWaves = 4;

// Sum or maximum over the four lanes of a column (l, l + 16, l + 32, l + 48).
__device__ __forceinline__ float column_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return other_half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float column_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return other_half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <bool BF16> __device__ __forceinline__ floatx4 mma16(floatx4 acc, const Frag<BF16> &a, const Frag<BF16> &b) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], acc, 0, 0, 0);
    return acc;
  }
}

// Cache rows are read once: nontemporal where a load takes whole lines.
template <class V> __device__ __forceinline__ V load_once(const char *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const V *>(p));
}

// 8 keys' pieces of D / 16 channels.
template <bool BF16, int D> struct Values {
  static constexpr int C = D / 16, W = BF16 ? C / 2 : C;  // channels and words of a piece
  uint32_t w[8][W];
  __device__ __forceinline__ void load(int j, const char *p) {
    if constexpr (W == 2) {
      const uintx2 x = load_once<uintx2>(p);
      w[j][0] = x[0];
      w[j][1] = x[1];
    } else {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uintx4 x = load_once<uintx4>(p + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][i + e] = x[e];
      }
    }
  }
  __device__ __forceinline__ void zero(int j) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[j][i] = 0;
  }
  // channel r of the 8 keys
  __device__ __forceinline__ Frag<BF16> block(int r) const {
    if constexpr (BF16) {
      uintx4 x;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        x[t] = __builtin_amdgcn_perm(w[2 * t + 1][r >> 1], w[2 * t][r >> 1], r & 1 ? 0x07060302u : 0x05040100u);
      return Frag<true>{__builtin_bit_cast(bf16x8, x)};
    } else {
      Frag<false> f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] = __uint_as_float(w[j][r]);
      return f;
    }
  }
};

__device__ __forceinline__ int length_of(const DecodeArgs &p, int n) {
  const int64_t most = p.P > 0 ? (int64_t)p.M * p.page : 0;
  const int len = p.lengths[n];
  return len < 0 ? 0 : (int)min((int64_t)len, most);
}
// The first key of the first span.
__device__ __forceinline__ int first_key(const DecodeArgs &p, int len) {
  return p.window && len > p.window ? (len - p.window) & ~(kTileKeys - 1) : 0;
}

// The workspace: maximum and sum of each head's spans, then (from a multiple of 16 bytes on) their outputs.
__host__ __device__ __forceinline__ int64_t outputs_at(int64_t N, int H, int splits) { return (N * H * splits * 2 + 3) & ~(int64_t)3; }

// ONE: a tile of 32 keys lies in one page.
template <bool BF16, int D, bool ONE>
__global__ void __launch_bounds__(256, BF16 || D == 64 ? 2 : 1) attention_decode_kernel(const DecodeArgs p, const DecodePlan plan, int shift) {
  using Vals = Values<BF16, D>;
  constexpr int ES = BF16 ? 2 : 4, C = Vals::C;
  __shared__ float part_o[kWaves][16][D + 4];
  __shared__ float part_m[kWaves][16], part_l[kWaves][16];
  const int units = p.N * p.Hkv * plan.tiles;
  const int split = blockIdx.x / units, unit = blockIdx.x % units;
  const int n = unit / (p.Hkv * plan.tiles), kv = unit / plan.tiles % p.Hkv, qt = unit % plan.tiles;
  const int group = p.H / p.Hkv, count = min(group - 16 * qt, 16);  // query heads of this workgroup
  const int head0 = kv * group + 16 * qt;
  const int len = length_of(p, n), lo = p.window ? max(len - p.window, 0) : 0;
  const int begin = first_key(p, len) + split * plan.span;
  if (split && begin >= len) return;
  const int end = min(len, begin + plan.span);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;

  Frag<BF16> q[D / 32];
  const int mine = min(col, count - 1);
#pragma unroll
  for (int kk = 0; kk < D / 32; ++kk) {
    const char *src = static_cast<const char *>(p.q) + (((int64_t)n * p.H + head0 + mine) * D + 32 * kk + 8 * g) * ES;
    if constexpr (BF16) {
      q[kk].v = *reinterpret_cast<const bf16x8 *>(src);
    } else {
      const floatx4 *f = reinterpret_cast<const floatx4 *>(src);
      q[kk].v = __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
  const float c = p.scale * kLog2e;
  const int32_t *table = p.pages + (int64_t)n * p.M;
  const char *kc = static_cast<const char *>(p.kc), *vc = static_cast<const char *>(p.vc);
  // the row of key `key` of page `page` in the cache, in values
  auto row_at = [&](int page, int key) { return (((int64_t)page * p.Hkv + kv) * p.page + (key & (p.page - 1))) * D; };

  // One tile on its way: keys as score operands, values, whether the keys of this lane's 8 slots are seen.
  struct Load {
    Frag<BF16> k[2][D / 32];
    Vals v;
    uint32_t seen;
  };
  // ONE: the page of the tile; else pages are looked up key by key
  auto page_of = [&](int key0) { return ONE && key0 < end ? table[__builtin_amdgcn_readfirstlane(key0 >> shift)] : -1; };
  auto load = [&](Load &x, int key0, int page) __attribute__((always_inline)) {
    int64_t kat[2], vat[8];
    x.seen = 0;
    if constexpr (ONE) {
      const bool there = page >= 0 && page < p.P;
      const int64_t base = row_at(there ? page : 0, key0);
#pragma unroll
      for (int u = 0; u < 2; ++u) kat[u] = base + (16 * u + col) * D;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = 16 * (j >> 2) + 4 * g + (j & 3);
        vat[j] = base + key * D;
        x.seen |= (uint32_t)(there && key0 + key >= lo && key0 + key < end) << j;
      }
    } else {
      const int most = p.M - 1;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = key0 + 16 * u + col, pg = table[min(key >> shift, most)];
        kat[u] = row_at(pg >= 0 && pg < p.P ? pg : 0, key);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 16 * (j >> 2) + 4 * g + (j & 3), pg = table[min(key >> shift, most)];
        const bool there = pg >= 0 && pg < p.P;
        vat[j] = row_at(there ? pg : 0, key);
        x.seen |= (uint32_t)(there && key >= lo && key < end) << j;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
        const char *src = kc + (kat[u] + 32 * kk + 8 * g) * ES;
        if constexpr (BF16) {
          x.k[u][kk].v = *reinterpret_cast<const bf16x8 *>(src);
        } else {
          const floatx4 *f = reinterpret_cast<const floatx4 *>(src);
          x.k[u][kk].v = __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7);
        }
      }
#pragma unroll
    for (int j = 0; j < 8; ++j) x.v.load(j, vc + (vat[j] + col * C) * ES);
  };

  floatx4 acc[C];
#pragma unroll
  for (int r = 0; r < C; ++r) acc[r] = zero4();
  float top = neg_inf(), sum = 0.f;
  auto take = [&](Load &x) __attribute__((always_inline)) {
    floatx4 s[2] = {zero4(), zero4()};
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
      for (int u = 0; u < 2; ++u) s[u] = mma16<BF16>(s[u], x.k[u][kk], q[kk]);
    // a lane's scores are of the keys of its 8 slots
    if (!__all(x.seen == 0xffu)) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!((x.seen >> j) & 1u)) {
          s[j >> 2][j & 3] = neg_inf();
          x.v.zero(j);  // whatever lies behind the last key
        }
    }
    float t = neg_inf();
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaxf(t, s[j >> 2][j & 3]);
    t = column_max(t) * c;
    if (__any(t > top + 8.f)) {  // as in the forward of whole sequences: nearly never after the first tile
      const bool grow = t > top + 8.f;
      const float f = grow ? __builtin_amdgcn_exp2f(top - t) : 1.f;
      top = grow ? t : top;
      sum *= f;
#pragma unroll
      for (int r = 0; r < C; ++r) acc[r] *= f;
    }
    const float base = top == neg_inf() ? 0.f : top;
    floatx8 w;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j >> 2][j & 3], c, -base));
      sum += w[j];
    }
    if constexpr (BF16) {
      // Probabilities in two parts of 8 bits each: the cache's reads bound the call, so that a second product costs nothing
      // (N4 131072 tokens 85.4 us with one rounded part, 85.9 so) and outputs are off by their own rounding alone (1.63e-3
      // of their norm, 2.3e-3 with one). The first is cut off, not rounded, so that what it leaves is not below zero; nor
      // is that zero unless all is, as an infinite value may meet neither.
      floatx8 first, rest;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        first[j] = __uint_as_float(__float_as_uint(w[j]) & 0xffff0000u);
        rest[j] = fmaxf(w[j] - first[j], fminf(w[j], 0x1p-126f));
      }
      const Frag<BF16> high{__builtin_convertvector(first, bf16x8)}, low{__builtin_convertvector(rest, bf16x8)};
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const Frag<BF16> v8 = x.v.block(r);
        acc[r] = mma16<BF16>(mma16<BF16>(acc[r], v8, low), v8, high);
      }
    } else {
#pragma unroll
      for (int r = 0; r < C; ++r) acc[r] = mma16<BF16>(acc[r], x.v.block(r), Frag<BF16>{w});
    }
  };

  // the next tile's loads are out before this one's are waited for, its page one tile earlier
  constexpr int STEP = kTileKeys * kWaves;
  int key0 = begin + kTileKeys * wave;
  if (key0 < end) {
    Load x[2];
    int page = page_of(key0), next = page_of(key0 + STEP);
    load(x[0], key0, page);
    for (;; key0 += 2 * STEP) {
      page = next;
      next = page_of(key0 + 2 * STEP);
      if (key0 + STEP < end) load(x[1], key0 + STEP, page);
      take(x[0]);
      if (key0 + STEP >= end) break;
      page = next;
      next = page_of(key0 + 3 * STEP);
      if (key0 + 2 * STEP < end) load(x[0], key0 + 2 * STEP, page);
      take(x[1]);
      if (key0 + 2 * STEP >= end) break;
    }
  }
  sum = column_sum(sum);

  // join the waves
  if (g == 0) {
    part_m[wave][col] = top;
    part_l[wave][col] = sum;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < C; r += 4)
      *reinterpret_cast<floatx4 *>(&part_o[wave][col][(4 * g + i) * C + r]) =
          floatx4{acc[r][i], acc[r + 1][i], acc[r + 2][i], acc[r + 3][i]};
  __syncthreads();
  constexpr int PER = D / 4;  // threads of a query: four channels each
  for (int x = tid; x < count * PER; x += 256) {
    const int qi = x / PER, d = x % PER * 4;
    float most = neg_inf(), l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) most = fmaxf(most, part_m[w][qi]);
    floatx4 o = zero4();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      // a wave that saw nothing: -inf on both sides, or a weight of zero
      const float f = part_m[w][qi] == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(part_m[w][qi] - most);
      l += f * part_l[w][qi];
      o += *reinterpret_cast<const floatx4 *>(&part_o[w][qi][d]) * f;
    }
    const int64_t at = (int64_t)n * p.H + head0 + qi;
    if (plan.splits == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const float y[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
      store_f<BF16, 4>(p.o, (size_t)(at * D + d), y);
    } else {
      float *ml = p.workspace + (at * plan.splits + split) * 2;
      float *to = p.workspace + outputs_at(p.N, p.H, plan.splits) + (at * plan.splits + split) * D + d;
      if (d == 0) {
        ml[0] = most;
        ml[1] = l;
      }
      *reinterpret_cast<floatx4 *>(to) = o;
    }
  }
}

// One workgroup a query head: its spans' sums, dealt out to WAVES waves, D / 64 neighbouring channels a lane.
template <bool BF16, int D, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) attention_decode_join_kernel(const DecodeArgs p, const DecodePlan plan) {
  constexpr int V = D / 64;
  __shared__ float sums[WAVES][D + 1];
  const int64_t at = blockIdx.x;
  const int n = (int)(at / p.H), len = length_of(p, n), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // span 0 is always written
  const int live = max(1, (len - first_key(p, len) + plan.span - 1) / plan.span);
  const float *ml = p.workspace + at * plan.splits * 2;
  const float *os = p.workspace + outputs_at(p.N, p.H, plan.splits) + at * plan.splits * D + V * lane;
  float most = neg_inf();
  for (int s = lane; s < live; s += 64) most = fmaxf(most, ml[2 * s]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) most = fmaxf(most, __shfl_xor(most, x));
  float o[V] = {}, l = 0.f;
#pragma unroll 4
  for (int s = wave; s < live; s += WAVES) {
    const float f = ml[2 * s] == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(ml[2 * s] - most);
    l += f * ml[2 * s + 1];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] += f * os[(int64_t)s * D + e];
  }
#pragma unroll
  for (int e = 0; e < V; ++e) sums[wave][V * lane + e] = o[e];
  if (lane == 0) sums[wave][D] = l;
  __syncthreads();
  const int d = threadIdx.x;
  if (d >= D) return;
  l = 0.f;
  float y[1] = {0.f};
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    l += sums[w][D];
    y[0] += sums[w][d];
  }
  y[0] *= l == 0.f ? 0.f : 1.f / l;
  store_f<BF16, 1>(p.o, (size_t)(at * D + d), y);
}

// ---------------------------------------------------------------- the cache's writes
// A wave a token: its place by its sequence's length and page table, then 16 bytes a lane.
__global__ void __launch_bounds__(256) kv_cache_store_kernel(const StoreArgs p, int shift) {
  const int lane = threadIdx.x & 63;
  const int es = p.bf16 ? 2 : 4, piece = p.d * es / 16, pieces = p.Hkv * piece;
  for (int64_t token = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); token < p.T; token += (int64_t)gridDim.x * 4) {
    int n = (int)token;
    int64_t behind = 1;  // tokens from this one to its sequence's end
    if (p.cu) {
      // the last sequence that begins at or before the token, by 64 tries at once
      int lo = 0, cnt = p.N;
      while (cnt > 1) {
        const int step = (cnt + 63) >> 6, i = lane * step;
        const uint64_t b = __ballot(i < cnt && p.cu[lo + min(i, cnt - 1)] <= token);
        const int c = b ? 63 - __builtin_clzll(b) : 0;
        lo += c * step;
        cnt = min(step, cnt - c * step);
      }
      n = lo;
      behind = p.cu[n + 1] - token;
      if (p.cu[n] > token || behind <= 0) continue;
    }
    const int64_t at = p.lengths[n] - behind;
    if (at < 0 || (at >> shift) >= p.M) continue;
    const int page = p.pages[(int64_t)n * p.M + (at >> shift)];
    if (page < 0 || page >= p.P) continue;
    const int64_t row = at & (p.page - 1);
    for (int i = lane; i < 2 * pieces; i += 64) {
      const bool v = i >= pieces;
      const int x = v ? i - pieces : i, hk = x / piece, c = x % piece;
      const char *from = static_cast<const char *>(v ? p.v : p.k) + (token * (v ? p.sv : p.sk) + (int64_t)hk * p.d) * es + c * 16;
      char *to = static_cast<char *>(v ? p.vc : p.kc) + ((((int64_t)page * p.Hkv + hk) << shift) + row) * p.d * es + c * 16;
      *reinterpret_cast<uintx4 *>(to) = *reinterpret_cast<const uintx4 *>(from);
    }
  }
}

int log2_of(int x) { return 31 - __builtin_clz((unsigned)x); }

template <bool BF16, int D> hipError_t run(const DecodeArgs &p, const DecodePlan &plan, hipStream_t stream) {
  const unsigned grid = (unsigned)((size_t)p.N * p.Hkv * plan.tiles * plan.splits);
  const int shift = log2_of(p.page);
  if (p.page >= kTileKeys) attention_decode_kernel<BF16, D, true><<<grid, 256, 0, stream>>>(p, plan, shift);
  else attention_decode_kernel<BF16, D, false><<<grid, 256, 0, stream>>>(p, plan, shift);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess || plan.splits == 1) return e;
  // few heads over many spans: 16 waves a head (N4 H16, 256 spans: 86 us in all against 88); many heads over few
  // spans: 4 (N256 H16, 4 spans: 208 against 220)
  const unsigned heads = (unsigned)((size_t)p.N * p.H);
  if (plan.splits > 32) attention_decode_join_kernel<BF16, D, 16><<<heads, 1024, 0, stream>>>(p, plan);
  else attention_decode_join_kernel<BF16, D, 4><<<heads, 256, 0, stream>>>(p, plan);
  return hipGetLastError();
}

}  // namespace

// A span is as long as leaves 2048 workgroups, 8 a CU, which even out sequences
// of different lengths (N256 up to 8192 tokens H16/2 d128 bf16: 208 us, 216 with
// 1024, 214 with 4096); 128 keys (a tile a wave) at least. Up to 512 keys are one span and
// one launch (N4 300 keys H32/4 d64: 6.1 us, 8.7 with three spans joined).
DecodePlan decode_plan(int N, int H, int Hkv, int M, int page, int window) {
  const int64_t all = (int64_t)M * page;
  // a window's keys begin inside a tile
  const int64_t most = window && window < all ? (window < all - kTileKeys ? window + kTileKeys : all) : all;
  DecodePlan plan;
  plan.tiles = (H / Hkv + 15) / 16;
  const int64_t units = (int64_t)N * Hkv * plan.tiles;
  int64_t span = most <= 512 ? 512 : 128;
  while (span < 4096 && units * ((most + 2 * span - 1) / (2 * span)) >= 2048) span *= 2;
  // nor more spans than a join has to be quick over
  while ((most + span - 1) / span > 1024) span *= 2;
  plan.span = (int)span;
  plan.splits = (int)(most > 0 ? (most + span - 1) / span : 1);
  return plan;
}

size_t decode_workspace_bytes(const DecodePlan &plan, int N, int H, int d) {
  return plan.splits == 1 ? 0 : ((size_t)outputs_at(N, H, plan.splits) + (size_t)N * H * plan.splits * d) * 4;
}

hipError_t launch_attention_decode(const DecodeArgs &p, hipStream_t stream) {
  const DecodePlan plan = decode_plan(p.N, p.H, p.Hkv, p.M, p.page, p.window);
  if (p.bf16) return p.d == 128 ? run<true, 128>(p, plan, stream) : run<true, 64>(p, plan, stream);
  return p.d == 128 ? run<false, 128>(p, plan, stream) : run<false, 64>(p, plan, stream);
}

hipError_t launch_kv_cache_store(const StoreArgs &p, hipStream_t stream) {
  const int64_t groups = ((int64_t)p.T + 3) / 4;
  kv_cache_store_kernel<<<(unsigned)(groups < 8192 ? groups : 8192), 256, 0, stream>>>(p, log2_of(p.page));
  return hipGetLastError();
}

}  // namespace gdn2
