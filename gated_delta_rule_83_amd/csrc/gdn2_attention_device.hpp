// gdn2_attention_device.hpp -- tiles, operands and masks that the attention
// kernels share (gfx950 only).
//
// Every product runs on 32 x 32 accumulators (lane l: column l & 31, half
// h = l >> 5; register i: row 8 (i / 4) + 4 h + i % 4) over steps of 16 of the
// contracted axis, whose operands hold 8 values a lane: row (A) or column (B)
// l & 31, values 8 h .. 8 h + 7 of the step. Two facts carry the kernels:
//  - an accumulator's registers 8 s .. 8 s + 7, read as rows of the contracted
//    axis, are already a B operand if the A operand takes the same order:
//    slot j is row 16 s + 8 (j / 4) + 4 h + j % 4. So scores become the next
//    product's operand in registers.
//  - a column of such an accumulator belongs to one lane (and its partner of
//    the other half): scores are kept transposed where a softmax row has to
//    be a column, so row statistics are sums over a lane's own registers.
// bf16 operands of columns of a tile come from LDS with transposing reads, so
// a tile lies there once, row by row.
#pragma once

#include "gdn2_attention.hpp"
#include "gdn2_vec.hpp"

namespace gdn2 {
namespace attn {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float floatx8 __attribute__((ext_vector_type(8)));
typedef short shortx8 __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = (float)(1.44269504088896341 - (double)kLog2e);
constexpr float kLn2 = 0.693147180559945309f, kLn2Low = (float)(0.693147180559945309 - (double)kLn2);

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Exponents of 2 for scale * s - base. In fp32 the factor scale * log2 e is kept
// in two parts: its rounding alone would show in every probability.
template <bool BF16> struct Exponent {
  float c, low;
  __device__ __forceinline__ explicit Exponent(float scale) {
    c = scale * kLog2e;
    low = BF16 ? 0.f : __builtin_fmaf(scale, kLog2eLow, __builtin_fmaf(scale, kLog2e, -c));
  }
  // base in powers of two
  __device__ __forceinline__ float operator()(float s, float base) const {
    const float x = __builtin_fmaf(s, c, -base);
    return BF16 || s == neg_inf() ? x : __builtin_fmaf(s, low, x);
  }
};

template <bool BF16> struct Frag;
template <> struct Frag<true> { bf16x8 v; };
template <> struct Frag<false> { floatx8 v; };

template <bool BF16> __device__ __forceinline__ floatx16 mma(floatx16 acc, const Frag<BF16> &a, const Frag<BF16> &b) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
  } else {
    // one step of 2 takes value j of both halves: 8 of them are a step of 16 in the same order
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], acc, 0, 0, 0);
    return acc;
  }
}

__device__ __forceinline__ floatx16 zero16() {
  floatx16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// registers 8 s .. 8 s + 7 of an accumulator as an operand
template <bool BF16> __device__ __forceinline__ Frag<BF16> operand(const floatx16 &x, int s) {
  floatx8 y;
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[8 * s + j];
  if constexpr (BF16) return Frag<true>{__builtin_convertvector(y, bf16x8)};
  else return Frag<false>{y};
}

// what an operand's rounding left of x
template <bool BF16> __device__ __forceinline__ Frag<BF16> remainder(const floatx16 &x, int s, const Frag<BF16> &w) {
  floatx16 y;
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = x[8 * s + j] - (float)w.v[j];
  return operand<BF16>(y, 0);
}

// acc += sum of N operands' products. In fp32 the sum of a tile is one of its
// own first: a chain over all of a long sequence would lose half a digit.
template <bool BF16, int N, class A> __device__ __forceinline__ void add_products(floatx16 &acc, A a, const Frag<BF16> (&b)[N]) {
  floatx16 t = BF16 ? acc : zero16();
#pragma unroll
  for (int i = 0; i < N; ++i) t = mma<BF16>(t, a(i), b[i]);
  if constexpr (BF16) acc = t;
  else acc += t;
}

// row of register i of a lane of half h
__device__ __forceinline__ constexpr int row_of(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// ---------------------------------------------------------------- tiles in LDS
// R rows of D values, 16-byte chunks exchanged within a row so that neither 16
// rows of one chunk nor 4 rows of 64 bytes meet in a bank.
template <bool BF16, int D> struct Tile {
  static constexpr int ES = BF16 ? 2 : 4, ROW = D * ES, CHUNKS = ROW / 16;
  static __device__ __forceinline__ int swizzle(int r) {
    if constexpr (CHUNKS >= 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return ((r & 2) << 1) | ((r >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int r, int chunk) { return r * ROW + ((chunk ^ swizzle(r)) << 4); }

};

template <class V> __device__ __forceinline__ V lds_read(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) const V *>((uintptr_t)at);
}

// A lane's places in a tile. Rows 16 apart are exchanged alike, so the places of
// rows r .. r + 15 serve all the others: what a read adds is a constant. `first`
// (a multiple of 32, below the tile's rows): the row that counts as row 0.
// LEAN (fp32): addresses are computed at every read; kept over a loop, as the compiler would, they take 2 registers a
// step and 8 a block.
template <bool BF16, int D, bool LEAN = false> struct Along {  // rows as rows or columns of an operand, contracted along them
  using L = Tile<BF16, D>;
  uint32_t off[BF16 ? D / 16 : 1];
  __device__ __forceinline__ void init(int lane, int first = 0) {
    const int r = lane & 31, h = lane >> 5;
    if constexpr (BF16) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) off[kk] = L::at(r, 2 * kk + h) + first * L::ROW;
    } else {
      off[0] = L::at(r, 2 * h) + first * L::ROW;  // step kk: chunk 4 kk on top, in bits of its own
    }
  }
  // row r0 + (lane & 31), values 16 kk + 8 h ..; tile: LDS address; r0 a multiple of 16
  __device__ __forceinline__ Frag<BF16> read(uint32_t tile, int r0, int kk) const {
    if constexpr (BF16) {
      return Frag<true>{lds_read<bf16x8>(off[kk] + (tile + r0 * L::ROW))};
    } else {
      uint32_t o = off[0];
      if constexpr (LEAN) pin_regs(o);
      o ^= (uint32_t)(4 * kk) << 4;
      const floatx4 x = lds_read<floatx4>(o + (tile + r0 * L::ROW)), y = lds_read<floatx4>((o ^ 16) + (tile + r0 * L::ROW));
      return Frag<false>{__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7)};
    }
  }
};

// Columns, contracted across the rows: slot j is row 8 (j / 4) + 4 h + j % 4.
// bf16: in a transposing read lane 4 a + b of 16 receives value b of the 8 bytes
// that lanes a, a + 4, a + 8 and a + 12 address, so lane j addresses row j / 4,
// columns 4 (j % 4).
template <bool BF16, int D, bool LEAN = false> struct Across {
  using L = Tile<BF16, D>;
  uint32_t off[D / 32][BF16 ? 2 : 1];
  __device__ __forceinline__ void init(int lane, int first = 0) {
    const int h = lane >> 5;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      if constexpr (BF16) {
        const int col = 32 * b + 16 * ((lane >> 4) & 1) + 4 * (lane & 3), r = 4 * h + ((lane >> 2) & 3);
#pragma unroll
        for (int e = 0; e < 2; ++e) off[b][e] = L::at(r + 8 * e, col >> 3) + 2 * (col & 7) + first * L::ROW;
      } else {
        const int col = 32 * b + (lane & 31);
        off[b][0] = L::at(4 * h, col >> 2) + 4 * (col & 3) + first * L::ROW;
      }
    }
  }
  // columns 32 b + (lane & 31), rows r0 .. r0 + 15
  __device__ __forceinline__ Frag<BF16> read(uint32_t tile, int r0, int b) const {
    const uint32_t at = tile + r0 * L::ROW;
    if constexpr (BF16) {
      auto rd = [&](uint32_t x) {
        return __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16 *)(uintptr_t)(x + at)));
      };
      return Frag<true>{__builtin_shufflevector(rd(off[b][0]), rd(off[b][1]), 0, 1, 2, 3, 4, 5, 6, 7)};
    } else {
      Frag<false> f;
      uint32_t x = off[b][0];
      if constexpr (LEAN) pin_regs(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        constexpr int ROW = L::ROW;
        const int r = 8 * (j >> 2) + (j & 3);  // on top of 4 h: bits of their own, in the exchange too
        f.v[j] = lds_read<float>((x ^ (L::swizzle(r) << 4)) + (at + r * ROW));
      }
      return f;
    }
  }
};

// ---------------------------------------------------------------- tiles from memory
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); }

// R rows straight from memory into a tile: 16 bytes a lane, which land in LDS
// in the order of the lanes; the exchange of chunks is in the addresses read.
// The wave-uniform part of an address is the buffer's base, so that a lane
// keeps one offset for all tiles. Rows past the last one are outside the
// buffer (zeros, or what the tile held); they are never visible. The compiler
// does not see these loads: landed() before the barrier that hands a tile over.
// 64 lanes' 16 (or 4) bytes at base + off, bounded by `bytes`, to LDS address `to` on.
template <int BYTES> __device__ __forceinline__ void dma(const char *base, uint32_t bytes, uint32_t off, uint32_t to) {
  const uintx4 rsrc = {uniform((uint32_t)(uintptr_t)base), uniform((uint32_t)((uintptr_t)base >> 32)) & 0xffffu, uniform(bytes),
                       0x00020000u};
  // Nothing else in these kernels uses m0. The compiler knows of no hazard inside the asm: one wait state between the
  // write of m0 and its use, five between a vector instruction's write of a scalar register (the descriptor's, by
  // readfirstlane) and a memory instruction's read of it.
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(uniform(to)), "v"(off), "s"(rsrc)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(uniform(to)), "v"(off), "s"(rsrc)
                 : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)static_cast<const char *>(p);
}

template <bool BF16, int D, int R, int THREADS = 256> struct Dma {
  using L = Tile<BF16, D>;
  static constexpr int N = R * L::CHUNKS / THREADS, RPI = THREADS / L::CHUNKS;  // rows of one turn
  static_assert(R * L::CHUNKS % THREADS == 0 && THREADS % L::CHUNKS == 0, "whole rows a turn");
  static constexpr int OFFS = RPI % 16 ? 16 / RPI : 1;  // turns after which the exchange repeats
  uint32_t off[OFFS], stride;
  // s: bytes between rows
  __device__ __forceinline__ void init(int64_t s, int tid) {
    stride = (uint32_t)s;
#pragma unroll
    for (int i = 0; i < OFFS; ++i) {
      const int r = tid / L::CHUNKS + i * RPI;
      off[i] = (tid / L::CHUNKS) * stride + (((tid % L::CHUNKS) ^ L::swizzle(r)) << 4);
    }
  }
  // base: row 0 of the sequence and head
  __device__ __forceinline__ void load(const char *tile, const char *base, int row0, int n, int wave) const {
    const uint32_t rows = (uint32_t)min(n - row0, R), to = lds_address(tile) + wave * 1024;
    const char *from = base + (int64_t)row0 * stride;
    // the whole offset in the lane's part: the bounds check does not hold for a uniform part past the end
#pragma unroll
    for (int i = 0; i < N; ++i)
      dma<16>(from, (rows - 1) * stride + L::ROW, off[i % OFFS] + i * RPI * stride, to + i * THREADS * 16);
  }
};
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Row `row` of a tensor as B operands of the steps along it (values 16 kk + 8 h ..).
template <bool BF16, int D> __device__ __forceinline__ void load_row(Frag<BF16> (&f)[D / 16], const char *row, int h) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    if constexpr (BF16) {
      f[kk].v = *reinterpret_cast<const bf16x8 *>(row + (16 * kk + 8 * h) * 2);
    } else {
      const floatx4 *p = reinterpret_cast<const floatx4 *>(row + (16 * kk + 8 * h) * 4);
      f[kk].v = __builtin_shufflevector(p[0], p[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
}

// The rows are there from here on. Left to itself the compiler waits for them where they are used first, inside
// the loop, and with them for the tile that is on its way.
template <class F, int N> __device__ __forceinline__ void arrived(F (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) pin_regs(f[i]);
}

// An accumulator of D / 32 blocks whose column is a row of the tensor at `row`, times f.
template <bool BF16, int D> __device__ __forceinline__ void store_row(char *row, const floatx16 (&acc)[D / 32], float f, int h) {
#pragma unroll
  for (int b = 0; b < D / 32; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const float x[4] = {acc[b][i] * f, acc[b][i + 1] * f, acc[b][i + 2] * f, acc[b][i + 3] * f};
      store_at<BF16, 4>(row + (32 * b + row_of(i, h)) * (BF16 ? 2 : 4), x);
    }
}

// ---------------------------------------------------------------- values in hidden places
// In a tile of which some places are hidden, an infinity or NaN there must leave
// nothing, though 0 times it is NaN, and one in a place that a row sees must
// reach that row's result in its column. A workgroup computes as if there
// were none; if a result is no number in the end (rare), it computes once more
// with such tiles' odd values replaced by zero (clean), then looks through those
// tiles again for the odd values that a result sees (restore): weighted by a
// probability, which is above zero, they are added as they are; weighted by a
// gradient of a score, NaN stands for them, as their scores are not finite.
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {  // sign bits of the bf16 halves that are no number
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
__device__ __forceinline__ bool odd(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; }

// Whether any of the workgroup's waves says so. `said`: a word of each.
template <int WAVES> __device__ __forceinline__ bool any_wave(bool f, uint32_t (&said)[WAVES], int tid) {
  const bool any = __any(f);
  if ((tid & 63) == 0) said[tid >> 6] = any;
  __syncthreads();
  uint32_t x = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) x |= said[w];
  return uniform(x) != 0;
}

// Zeros for a tile's odd values. The whole workgroup calls, and nobody reads the tile meanwhile.
template <bool BF16, int BYTES> __device__ __forceinline__ void clean(char *t, int tid) {
#pragma unroll 1
  for (int i = tid * 16; i < BYTES; i += blockDim.x * 16) {
    uintx4 w = *reinterpret_cast<const uintx4 *>(t + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) w[j] &= ~((odd_halves(w[j]) >> 15) * 0xffffu);
      else if (odd(w[j])) w[j] = 0;
    }
    *reinterpret_cast<uintx4 *>(t + i) = w;
  }
  __syncthreads();
}

template <int N> __device__ __forceinline__ bool any_odd(const floatx16 (&acc)[N]) {
  bool f = false;
#pragma unroll
  for (int b = 0; b < N; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) f |= odd(__float_as_uint(acc[b][i]));
  return f;
}

// Rows first .. last of the tile are those this lane's column sees. ADD: the values themselves, else NaN.
template <bool BF16, int D, int R, bool ADD>
__device__ __forceinline__ void restore(floatx16 (&acc)[D / 32], const char *t, int first, int last, int h) {
  using L = Tile<BF16, D>;
  first = max(first, 0);
  last = min(last, R - 1);
#pragma unroll 1
  for (int r = first; r <= last; ++r)
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int col = 32 * b + row_of(i, h);  // 4 neighbouring values of the row
        if constexpr (BF16) {
          const uintx2 w = *reinterpret_cast<const uintx2 *>(t + L::at(r, col >> 3) + 2 * (col & 7));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16;
            if (odd(x)) acc[b][i + e] = ADD ? acc[b][i + e] + __uint_as_float(x) : __builtin_nanf("");
          }
        } else {
          const uintx4 w = *reinterpret_cast<const uintx4 *>(t + L::at(r, col >> 2));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (odd(w[e])) acc[b][i + e] = ADD ? acc[b][i + e] + __uint_as_float(w[e]) : __builtin_nanf("");
        }
      }
}

// ---------------------------------------------------------------- sequences and blocks
// Query i of n_q sees key j of n_k if lo(i) <= j <= hi(i), its own place on the
// key axis being i + n_k - n_q.
struct Mask {
  int nq, nk, shift, window;
  bool causal;
  __device__ __forceinline__ int hi(int i) const { return causal ? min(i + shift, nk - 1) : nk - 1; }
  __device__ __forceinline__ int lo(int i) const {
    return window ? (int)max((int64_t)i + shift - window + 1, (int64_t)0) : 0;
  }
  // the queries that see key j: first .. last
  __device__ __forceinline__ int first(int j) const { return causal ? (int)max((int64_t)j - shift, (int64_t)0) : 0; }
  __device__ __forceinline__ int last(int j) const {
    return window ? (int)min((int64_t)j - shift + window - 1, (int64_t)nq - 1) : nq - 1;
  }
};

__device__ __forceinline__ int clamp_to(int x, int T) { return x < 0 ? 0 : (x > T ? T : x); }

// Packed sequences: block slots s of sequence n are cu[n] / ROWS + n .. , which
// leaves every sequence room for its ragged last block; the workgroup finds n
// by 64 tries at once.
template <int ROWS>
__device__ __forceinline__ bool find_block(const int32_t *cu, int B, int T, int s, int *seq, int *row0) {
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = B;
  while (cnt > 1) {
    const int step = (cnt + 63) >> 6, i = lane * step;
    const bool below = i < cnt && clamp_to(cu[lo + min(i, cnt - 1)], T) / ROWS + lo + i <= s;
    const uint64_t b = __ballot(below);
    const int c = b ? 63 - __builtin_clzll(b) : 0;
    lo = __builtin_amdgcn_readfirstlane(lo + c * step);
    cnt = min(step, cnt - c * step);
    cnt = __builtin_amdgcn_readfirstlane(cnt);
  }
  *seq = lo;
  *row0 = (s - (clamp_to(cu[lo], T) / ROWS + lo)) * ROWS;
  return *row0 >= 0;
}

// Neighbouring workgroups go to the 8 dies in turn. Blocks run from the one that sees most on, over all heads: the
// longest first, so that the end is even. Where the heads (of all sequences) divide by 8, a die takes heads that
// share keys, whose tiles its L2 then holds; otherwise they are dealt out as they come.
__device__ __forceinline__ void find_work(unsigned units, unsigned *unit, unsigned *rank) {
  const unsigned i = blockIdx.x % units;
  *rank = blockIdx.x / units;
  *unit = units % 8 ? i : (i & 7) * (units >> 3) + (i >> 3);
}

// The rank'th block of packed sequences, from the one with the most to do on: find_block takes the last sequence
// first, and a long one near the front is begun when the rest is nearly done. For causal attention of up to 64
// sequences the blocks are counted by level instead (KEYS: of keys, whose first block is seen by most queries; else of
// queries, whose last block sees most keys, the prefix included): lane n holds sequence n's blocks nb and its lowest
// level c, and the level that the rank falls into is found by halves. us before / so, forward and backward: 8 sequences of
// 32768 tokens H8/2 d64, the longest 6266, 250 / 212 and 838 / 723; 24 of 16384 H16/4 d128, the longest 3147, 144 / 143
// and 556 / 507, the longest 2044, 132 / 121 and 459 / 431, the longest 1469, 119 / 124 and 453 / 428; 64 of 32768 H16/2
// d128, the longest 1967, 219 / 225 and 820 / 737: where all are short the forward loses 3%, less than the backward
// of the same sequences gains.
template <int ROWS, bool KEYS>
__device__ __forceinline__ bool find_ranked(const AttentionArgs &p, int slots, int rank, int *seq, int *row0) {
  const int32_t *cu = KEYS ? p.cu_k : p.cu_q;
  const int T = KEYS ? p.Tk : p.Tq;
  if (!p.causal || p.window || p.B > 64) return find_block<ROWS>(cu, p.B, T, KEYS ? rank : slots - 1 - rank, seq, row0);
  const int lane = threadIdx.x & 63;
  int nb = 0, c = 0;
  if (lane < p.B) {
    const int n = max(clamp_to(cu[lane + 1], T) - clamp_to(cu[lane], T), 0);
    nb = n / ROWS + (n % ROWS != 0);
    if (!KEYS && p.cu_k != p.cu_q) {
      const int nk = max(clamp_to(p.cu_k[lane + 1], p.Tk) - clamp_to(p.cu_k[lane], p.Tk), 0);
      c = max(nk - n, 0) / ROWS;
    }
  }
  // blocks of level x and above: a wave's sum
  auto count = [&](int x) {
    int sum = min(max(nb + c - x, 0), nb);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x111, 0xf, 0xf, true);  // lanes of a row of 16, 1, 2, 4, 8 apart
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x112, 0xf, 0xf, true);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x114, 0xf, 0xf, true);
    sum += __builtin_amdgcn_update_dpp(0, sum, 0x118, 0xf, 0xf, true);
    return __builtin_amdgcn_readlane(sum, 15) + __builtin_amdgcn_readlane(sum, 31) + __builtin_amdgcn_readlane(sum, 47) +
           __builtin_amdgcn_readlane(sum, 63);
  };
  if (count(0) <= rank) return false;  // no more blocks
  // the highest level that has the rank'th block at or above it
  int at = 0;
  for (int step = 1 << (31 - __builtin_clz((unsigned)(((int64_t)p.Tq + p.Tk) / ROWS) + 1u)); step; step >>= 1)
    if (count(at + step) > rank) at += step;
  const int left = rank - count(at + 1);
  const bool on = at >= c && at < c + nb;
  const uint64_t all = __ballot(on);
  const int n = __builtin_ctzll(__ballot(on && __builtin_popcountll(all & ((1ull << lane) - 1)) == left));
  const int block = at - __builtin_amdgcn_readlane(c, n);
  *seq = n;
  *row0 = (KEYS ? __builtin_amdgcn_readlane(nb, n) - 1 - block : block) * ROWS;
  return true;
}

// A sequence's tokens: the first query and key over the whole batch, how many there are, and
// the first of `head`'s values of a [head, query] array (lse, delta).
struct Span {
  int64_t q0, k0, rows;
  Mask m;
};
// unit: b * heads + head (batch) or head (packed, sequence seq)
__device__ __forceinline__ Span span_of(const AttentionArgs &p, int seq, int head) {
  Span s;
  s.m.causal = p.causal;
  s.m.window = p.window;
  if (p.cu_q) {
    const int a = clamp_to(p.cu_q[seq], p.Tq), b = clamp_to(p.cu_q[seq + 1], p.Tq);
    const int c = clamp_to(p.cu_k[seq], p.Tk), d = clamp_to(p.cu_k[seq + 1], p.Tk);
    s.m.nq = max(b - a, 0);
    s.m.nk = max(d - c, 0);
    s.q0 = a;
    s.k0 = c;
    s.rows = (int64_t)head * p.Tq + a;
  } else {
    s.m.nq = p.Tq;
    s.m.nk = p.Tk;
    s.q0 = (int64_t)seq * p.Tq;
    s.k0 = (int64_t)seq * p.Tk;
    s.rows = ((int64_t)seq * p.H + head) * p.Tq;
  }
  s.m.shift = s.m.nk - s.m.nq;
  return s;
}

// x combined with the other half's lane
__device__ __forceinline__ float other_half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace attn
}  // namespace gdn2
