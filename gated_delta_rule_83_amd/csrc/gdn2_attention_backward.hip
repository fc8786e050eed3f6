// gdn2_attention_backward.hip -- gradients of softmax attention.
//
//   p_ij = exp(s_ij - lse_i)     dv_j = sum_i p_ij dO_i     dp_ij = dO_i . v_j
//   delta_i = dO_i . o_i         ds_ij = p_ij (dp_ij - delta_i)
//   dq_i = scale sum_j ds_ij k_j              dk_j = scale sum_i ds_ij q_i
//
// Two passes, each of which computes the scores and dp again: one by blocks of
// queries (dq; it also leaves delta and lse for the other),
// one by blocks of keys (dk, dv, over the query heads that share them). That is
// 14 d flops a pair instead of the 10 d of a single pass, whose dq would have to
// be summed by atomics in an order of their own: here results are the same bits
// at every run. Scores are kept so that the rows of the product to come are the
// registers: keys for dq, queries for dk and dv.
//
// bf16 operands of the last products: p and ds are rounded once, 2^-8 at most,
// which is the size of the results' own rounding. In tiles of which some places
// are hidden (the diagonal's: there rows see few keys, and the largest
// probabilities are) the remainder goes through the product as well: gradients
// of 4096 causal tokens are 1.25 times as far off as their own rounding, of 200
// tokens 1.06 times, where one operand leaves 1.45 and 1.47; it costs 2% (B4
// T4096 H16/2 d128: 984 -> 1005 us).
//
// A query that sees one key has p = 1 and delta = dp: ds is zero (or NaN), of
// which two orders of the sums would leave noise, with nothing beside it where
// every query sees one. So dq's row, or all of dk, is multiplied by zero in the
// end; where one query does, the first key's own, its ds is in dk (in a partly
// hidden tile, the only kind that can hold it).
#include "gdn2_attention_device.hpp"

namespace gdn2 {
namespace {

using namespace attn;

// A row's lse in powers of two; in fp32 in two parts, as the factor of its scores.
// A row without any weight (lse -inf) has probabilities of zero, as +inf makes them.
__device__ __forceinline__ float base_of(float lse) { return lse == neg_inf() ? -lse : lse; }

template <bool BF16> struct Base {
  float high, low;
  Base() = default;
  __device__ __forceinline__ explicit Base(float lse) {
    *this = at(BF16 ? base_of(lse) * kLog2e : base_of(lse));
    pin_regs(high);
  }
  // from what the first pass leaves: powers of two in bf16, base_of(lse) in fp32
  static __device__ __forceinline__ Base at(float left) {
    Base b;
    if constexpr (BF16) {
      b.high = left;
      b.low = 0.f;
    } else {
      b.high = left * kLog2e;
      b.low = left == -neg_inf() ? 0.f : __builtin_fmaf(left, kLog2eLow, __builtin_fmaf(left, kLog2e, -b.high));
    }
    return b;
  }
  __device__ __forceinline__ float probability(const Exponent<BF16> &power, float s) const {
    const float x = power(s, high);
    return __builtin_amdgcn_exp2f(BF16 ? x : x - low);
  }
};

// ---------------------------------------------------------------- dq
// SPLIT 2: 64 queries a workgroup, each 32 on two waves with half of a tile's keys
// each, as in the forward where blocks are few (us: B1 T2048 H8/2 d128 bf16,
// the whole backward, 129 / 107, fp32 1062 / 891; B2 T1003 H6/3 d64 fp32 window
// 300 99 / 74).
template <bool BF16, int D, int SPLIT>
__global__ void __launch_bounds__(256, BF16 || D == 64 ? 2 : 1) attention_dq_kernel(const AttentionArgs p, unsigned units) {
  using L = Tile<BF16, D>;
  constexpr int ROWS = kAttnRows / SPLIT, PAIRS = 4 / SPLIT;
  constexpr int KT = BF16 || SPLIT == 2 ? 64 : 32, SUB = KT / 32 / SPLIT, ES = BF16 ? 2 : 4, TILE = KT * L::ROW;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[2][2][TILE];
    uint32_t said[4];
    float delta[SPLIT == 2 ? 4 : 1][64];
  } sm;
  unsigned unit, rank;
  find_work(units, &unit, &rank);
  const int slots = (int)(gridDim.x / units), tile = slots - 1 - (int)rank;  // causal: the last block sees most
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int seq, row0, head;
  if (p.cu_q) {
    if (!find_ranked<ROWS, false>(p, slots, (int)rank, &seq, &row0)) return;
    head = (int)unit;
  } else {
    seq = (int)(unit / (unsigned)p.H);
    head = (int)(unit % (unsigned)p.H);
    row0 = tile * ROWS;
  }
  const Span sp = span_of(p, seq, head);
  const Mask m = sp.m;
  if (row0 >= m.nq) return;
  const int kv = head / (p.H / p.Hkv);
  const char *kbase = static_cast<const char *>(p.k) + (sp.k0 * p.sk + (int64_t)kv * D) * ES;
  const char *vbase = static_cast<const char *>(p.v) + (sp.k0 * p.sv + (int64_t)kv * D) * ES;

  const int side = SPLIT == 1 ? 0 : wave / PAIRS, half = side * 32 * SUB;  // of the tiles' keys, from the half'th on
  const int mine = row0 + 32 * (wave % PAIRS) + (lane & 31), row = min(mine, m.nq - 1), hi = m.hi(row), lo = m.lo(row);
  const int64_t place = ((sp.q0 + row) * (int64_t)p.H + head) * D * ES;  // the row in o, dO and dq
  Frag<BF16> q[D / 16], g[D / 16];
  load_row<BF16, D>(q, static_cast<const char *>(p.q) + ((sp.q0 + row) * p.sq + (int64_t)head * D) * ES, h);
  load_row<BF16, D>(g, static_cast<const char *>(p.dO) + place, h);
  float delta = 0.f;
  {
    Frag<BF16> o[D / 16];
    load_row<BF16, D>(o, static_cast<const char *>(p.o_in) + place, h);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = __builtin_fmaf((float)o[kk].v[j], (float)g[kk].v[j], delta);
    delta = other_half_sum(delta);
  }
  arrived(q);
  arrived(g);
  const Exponent<BF16> power(p.scale);
  const Base<BF16> lse(p.lse_in[sp.rows + row]);
  const int blast = min(row0 + ROWS - 1, m.nq - 1);
  const int t_lo = m.lo(row0) / KT, t_hi = (m.hi(blast) + KT) / KT;
  const int b_lo = m.lo(blast), b_hi = m.hi(row0);
  auto hides = [&](int key0) { return key0 < b_lo || key0 + KT - 1 > b_hi; };

  floatx16 acc[D / 32];
  Along<BF16, D> along;
  Across<BF16, D> across;
  along.init(lane, half);
  across.init(lane, half);
  const uint32_t at = lds_address(&sm);  // tile [i][j] from (2 i + j) TILE on
  Dma<BF16, D, KT> ks, vs;
  ks.init(p.sk * ES, tid);
  vs.init(p.sv * ES, tid);

  const int most = m.window ? min(m.window, m.hi(blast) + 1) : m.hi(blast) + 1;  // keys that a query sees at most
  // delta from o as it was rounded is off by half a step of o, which shows where a query sees few keys and ds is
  // itself a difference of their size (1024 causal tokens: dq 1.6 times as far off as its own rounding, 1.43 with
  // the sum in fp32). There delta is summed from the probabilities instead: two products more, for five tiles at most.
  if (BF16 && t_lo < t_hi && most <= 128) {
    float own = 0.f;
#pragma unroll 1
    for (int t = t_lo; t < t_hi; ++t) {
      __syncthreads();  // nobody reads the tile before any more
      ks.load(sm.tile[0][0], kbase, t * KT, m.nk, wave);
      vs.load(sm.tile[0][1], vbase, t * KT, m.nk, wave);
      landed();
      __syncthreads();
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        floatx16 s = zero16(), dp = zero16();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          s = mma<BF16>(s, along.read(at, 32 * u, kk), q[kk]);
          dp = mma<BF16>(dp, along.read(at + TILE, 32 * u, kk), g[kk]);
        }
        const int from = lo - t * KT - half - 4 * h, to = hi - t * KT - half - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          own += 32 * u + row_of(i, 0) < from || 32 * u + row_of(i, 0) > to ? 0.f : lse.probability(power, s[i]) * dp[i];
      }
    }
    delta = other_half_sum(own);
    if constexpr (SPLIT == 2) sm.delta[wave][lane] = delta;
    __syncthreads();
    if constexpr (SPLIT == 2) delta += sm.delta[(wave + PAIRS) % 4][lane];
  }
  delta += 0.f * delta;  // of an infinite dO: NaN, whatever of dp - delta the dk, dv pass would make of it
  if (mine < m.nq && h == 0 && side == 0) {
    p.delta[sp.rows + mine] = delta;
    p.lse[sp.rows + mine] = BF16 ? lse.high : base_of(p.lse_in[sp.rows + mine]);
  }

  // ds of 32 keys
  auto part = [&](Frag<BF16> (&ds)[2], Frag<BF16> (&rest)[2], uint32_t kt, uint32_t vt, int u, int key0, auto masked) __attribute__((always_inline)) {
    floatx16 s = zero16(), dp = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      s = mma<BF16>(s, along.read(kt, 32 * u, kk), q[kk]);
      dp = mma<BF16>(dp, along.read(vt, 32 * u, kk), g[kk]);
    }
    const int from = lo - key0 - 4 * h, to = hi - key0 - 4 * h;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = lse.probability(power, s[i]) * (dp[i] - delta);
      if constexpr (decltype(masked)::value)
        if (32 * u + row_of(i, 0) < from || 32 * u + row_of(i, 0) > to) s[i] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      ds[e] = operand<BF16>(s, e);
      if constexpr (BF16 && decltype(masked)::value) rest[e] = remainder<BF16>(s, e, ds[e]);
    }
  };
  auto product = [&](const Frag<BF16> (&ds)[2], const Frag<BF16> (&rest)[2], uint32_t kt, int u, auto masked) __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(1);
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          const Frag<BF16> x = across.read(kt, 32 * u + 16 * e, b);
          acc[b] = mma<BF16>(acc[b], x, ds[e]);
          if constexpr (decltype(masked)::value) acc[b] = mma<BF16>(acc[b], x, rest[e]);
        }
    } else {
#pragma unroll
      for (int b = 0; b < D / 32; ++b) add_products<BF16>(acc[b], [&](int e) { return across.read(kt, 32 * u + 16 * e, b); }, ds);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  for (bool careful = false;; careful = true) {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) acc[b] = zero16();
    if (t_lo >= t_hi) break;
    ks.load(sm.tile[0][0], kbase, t_lo * KT, m.nk, wave);
    vs.load(sm.tile[0][1], vbase, t_lo * KT, m.nk, wave);
    auto turn = [&](int t, auto buf) __attribute__((always_inline)) {
      constexpr int BUF = decltype(buf)::value;
      const int key0 = t * KT;
      landed();
      __syncthreads();  // tile t is there, and nobody reads tile t - 1 any more
      if (t + 1 < t_hi) {
        ks.load(sm.tile[BUF ^ 1][0], kbase, key0 + KT, m.nk, wave);
        vs.load(sm.tile[BUF ^ 1][1], vbase, key0 + KT, m.nk, wave);
      }
      const uint32_t kt = at + 2 * BUF * TILE, vt = kt + TILE;
      Frag<BF16> ds[SUB][2], rest[SUB][2];
      if (hides(key0)) {
#pragma unroll
        for (int u = 0; u < SUB; ++u) part(ds[u], rest[u], kt, vt, u, key0 + half, std::true_type{});
        if (careful) {  // the scores take K as it is, the product without its odd values
          __syncthreads();
          clean<BF16, TILE>(sm.tile[BUF][0], tid);
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u) product(ds[u], rest[u], kt, u, std::true_type{});
      } else {
        // each 32 keys' product beside the next ones' scores
        part(ds[0], rest[0], kt, vt, 0, key0 + half, std::false_type{});
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          if (u + 1 < SUB) part(ds[u + 1], rest[u + 1], kt, vt, u + 1, key0 + half, std::false_type{});
          product(ds[u], rest[u], kt, u, std::false_type{});
        }
      }
    };
    for (int t = t_lo; t < t_hi; t += 2) {
      turn(t, std::integral_constant<int, 0>{});
      if (t + 1 < t_hi) turn(t + 1, std::integral_constant<int, 1>{});
    }
    if (careful) {
#pragma unroll 1
      for (int t = t_lo; t < t_hi; ++t) {
        if (!hides(t * KT)) continue;
        __syncthreads();
        ks.load(sm.tile[0][0], kbase, t * KT, m.nk, wave);
        landed();
        __syncthreads();
        restore<BF16, D, KT, false>(acc, sm.tile[0][0], lo - t * KT, hi - t * KT, h);
      }
      break;
    }
    if (!any_wave(any_odd(acc), sm.said, tid)) break;
  }
  if constexpr (SPLIT == 2) {  // the second half's sums into the first's, through what was the tiles' memory
    floatx4 *to = reinterpret_cast<floatx4 *>(&sm) + (wave % PAIRS) * (D / 32 * 4) * 64 + lane;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (side) to[(4 * b + i) * 64] = floatx4{acc[b][4 * i], acc[b][4 * i + 1], acc[b][4 * i + 2], acc[b][4 * i + 3]};
    __syncthreads();
    if (side) return;
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[b][i] += to[(4 * b + i / 4) * 64][i % 4];
  }
  if (mine < m.nq) store_row<BF16, D>(static_cast<char *>(p.dq) + place, acc, lo == hi ? 0.f : p.scale, h);
}

// ---------------------------------------------------------------- dk, dv
// 128 or 64 keys, 32 a pair of waves. The one keeps K and dv: scores, probabilities,
// dv += dO^T p; the other V and dk: dp, ds, dk += Q^T ds, one tile of queries
// behind, with the probabilities from LDS (in fp32: a rounding of them would
// stand beside the one of ds). So both have two products a tile and registers
// for two waves a SIMD, one of each kind; with all four products and both
// accumulators in one wave there is one a SIMD, whose vector instructions keep
// the matrix cores waiting (B4 T4096 H16/2 d128 bf16: 1061 us, so 640 to 674).
template <bool BF16, int D, int KEYS>
__global__ void __launch_bounds__(4 * KEYS, 2) attention_dkv_kernel(const AttentionArgs p, unsigned units) {
  using L = Tile<BF16, D>;
  constexpr int PAIRS = KEYS / 32, HALF = 64 * PAIRS;  // pairs of waves; threads of each kind
  constexpr int QT = 32, ES = BF16 ? 2 : 4, TILE = QT * L::ROW, RING = 3;
  constexpr int PROBS = 32 * 32 * 4;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[RING][2][TILE];  // Q, dO
    float stat[RING][2][64];   // lse in powers of two and delta of a tile's rows (64 lanes land, 32 are used)
    char probs[RING][PAIRS][PROBS];
    uint32_t said[2 * PAIRS];
  } sm;
  unsigned unit, rank;
  find_work(units, &unit, &rank);
  const int tile = (int)rank;  // causal: the first keys are seen most
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool second = wave >= PAIRS;  // keeps V and dk
  const int pair = wave % PAIRS;
  const int group = p.H / p.Hkv, share = group / p.parts;  // query heads of a key head, and of this workgroup
  int seq, row0;
  const int slice = (int)(unit % (unsigned)p.parts);
  unsigned kvu = unit / (unsigned)p.parts;
  if (p.cu_q) {
    if (!find_ranked<KEYS, true>(p, 0, tile, &seq, &row0)) return;
  } else {
    seq = (int)(kvu / (unsigned)p.Hkv);
    kvu %= (unsigned)p.Hkv;
    row0 = tile * KEYS;
  }
  const int kv = (int)kvu, head0 = kv * group + slice * share;
  const Span sp = span_of(p, seq, head0);
  const Mask m = sp.m;
  if (row0 >= m.nk) return;

  const int mine = row0 + 32 * pair + (lane & 31), row = min(mine, m.nk - 1);
  Frag<BF16> kept[D / 16];
  load_row<BF16, D>(kept, static_cast<const char *>(second ? p.v : p.k) + ((sp.k0 + row) * (second ? p.sv : p.sk) + (int64_t)kv * D) * ES, h);
  arrived(kept);
  const Exponent<BF16> power(p.scale);
  const int first = m.first(row), last = m.last(row);
  // query tiles that some key of the workgroup is seen from; queries that see every one of them
  const int blast = min(row0 + KEYS - 1, m.nk - 1);
  const int t_lo = m.first(row0) / QT, t_hi = (m.last(blast) + QT) / QT;
  const int b_lo = m.first(blast), b_hi = m.last(row0);
  auto hides = [&](int q0) { return q0 < b_lo || q0 + QT - 1 > b_hi; };
  const bool all_lone = m.nk == 1 || m.window == 1;  // every query sees one key
  const int lone = m.causal ? -m.shift : -1;         // else the query that does

  floatx16 acc[D / 32];
  constexpr bool LEAN = !BF16 && D == 128;
  Along<BF16, D, LEAN> along;
  Across<BF16, D, LEAN> across;
  along.init(lane);
  across.init(lane);
  const uint32_t at = lds_address(&sm), stats = lds_address(&sm.stat), probs = lds_address(&sm.probs) + pair * PROBS + lane * 16;
  const int nt = t_hi - t_lo, turns = nt > 0 ? nt * share : 0;
  // the first waves fetch Q, the second dO
  Dma<BF16, D, QT, HALF> rows;
  rows.init((second ? (int64_t)p.H * D : p.sq) * ES, tid % HALF);
  const char *base = second ? static_cast<const char *>(p.dO) + (sp.q0 * (int64_t)p.H + head0) * D * ES
                            : static_cast<const char *>(p.q) + (sp.q0 * p.sq + (int64_t)head0 * D) * ES;
  // tile t of head head0 + hd into buffer `to`
  auto fetch = [&](int hd, int t, int to) __attribute__((always_inline)) {
    const int r0 = t * QT;
    rows.load(sm.tile[to][second], base + (int64_t)hd * D * ES, r0, m.nq, pair);
    if (pair == 0) {
      const float *from = (second ? p.delta : p.lse) + sp.rows + (int64_t)hd * p.Tq + r0;
      dma<4>(reinterpret_cast<const char *>(from), (uint32_t)min(m.nq - r0, QT) * 4, lane * 4, lds_address(sm.stat[to][second]));
    }
  };
  // whether the query of register i does not see this lane's key
  auto outside = [&](int q0, int i) {
    const int from = first - q0 - 4 * h, to = last - q0 - 4 * h;
    return row_of(i, 0) < from || row_of(i, 0) > to;
  };

  // operands are read as they are used; read ahead, they do not fit the registers (B2 T4096 H8/2 fp32: backward
  // 3.9 ms with 265 registers spilled, 2.5 without)
  auto in_turn = [] {
    if constexpr (LEAN) __builtin_amdgcn_sched_barrier(0);
  };
  auto scores = [&](int q0, int buf, auto masked) __attribute__((always_inline)) {
    const uint32_t qt = at + 2 * buf * TILE, gt = qt + TILE, st = stats + buf * 512 + 16 * h, pt = probs + buf * PAIRS * PROBS;
    floatx16 s = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      s = mma<BF16>(s, along.read(qt, 0, kk), kept[kk]);
      in_turn();
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const floatx4 l = lds_read<floatx4>(st + 4 * row_of(i, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i + e] = Base<BF16>::at(l[e]).probability(power, s[i + e]);
    }
    if constexpr (decltype(masked)::value) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (outside(q0, i)) s[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<__attribute__((address_space(3))) floatx4 *>((uintptr_t)(pt + i * 256)) = floatx4{s[i], s[i + 1], s[i + 2], s[i + 3]};
    const Frag<BF16> w[2] = {operand<BF16>(s, 0), operand<BF16>(s, 1)};
    __builtin_amdgcn_s_setprio(1);
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        Frag<BF16> rest;
        if constexpr (decltype(masked)::value) rest = remainder<BF16>(s, e, w[e]);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          const Frag<BF16> x = across.read(gt, 16 * e, b);
          acc[b] = mma<BF16>(acc[b], x, w[e]);
          if constexpr (decltype(masked)::value) acc[b] = mma<BF16>(acc[b], x, rest);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        add_products<BF16>(acc[b], [&](int e) { return across.read(gt, 16 * e, b); }, w);
        in_turn();
      }
    }
    __builtin_amdgcn_s_setprio(0);
  };
  auto slopes = [&](int q0, int buf, auto masked) __attribute__((always_inline)) {
    const uint32_t qt = at + 2 * buf * TILE, gt = qt + TILE, st = stats + buf * 512 + 256 + 16 * h, pt = probs + buf * PAIRS * PROBS;
    floatx16 s = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      s = mma<BF16>(s, along.read(gt, 0, kk), kept[kk]);
      in_turn();
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const floatx4 d = lds_read<floatx4>(st + 4 * row_of(i, 0)), w = lds_read<floatx4>(pt + i * 256);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool alone = decltype(masked)::value && row_of(i, 0) + e == lone - q0 - 4 * h;
        s[i + e] = (alone ? 0.f : w[e]) * (s[i + e] - d[e]);
      }
    }
    if constexpr (decltype(masked)::value) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (outside(q0, i)) s[i] = 0.f;
    }
    const Frag<BF16> w[2] = {operand<BF16>(s, 0), operand<BF16>(s, 1)};
    __builtin_amdgcn_s_setprio(1);
    if constexpr (BF16) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        Frag<BF16> rest;
        if constexpr (decltype(masked)::value) rest = remainder<BF16>(s, e, w[e]);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          const Frag<BF16> x = across.read(qt, 16 * e, b);
          acc[b] = mma<BF16>(acc[b], x, w[e]);
          if constexpr (decltype(masked)::value) acc[b] = mma<BF16>(acc[b], x, rest);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        add_products<BF16>(acc[b], [&](int e) { return across.read(qt, 16 * e, b); }, w);
        in_turn();
      }
    }
    __builtin_amdgcn_s_setprio(0);
  };

  for (bool careful = false;; careful = true) {
#pragma unroll
    for (int b = 0; b < D / 32; ++b) acc[b] = zero16();
    if (turns == 0) break;
    fetch(0, t_lo, 0);
    // turn i: tile i for the first wave of a pair, tile i - 1 for the second; tile i + 1 on its way. Each kind has
    // a loop of its own with the same barriers.
    auto walk = [&](auto kind) __attribute__((always_inline)) {
      constexpr bool SECOND = decltype(kind)::value;
      int t = t_lo, ahead_hd = 0, ahead = t_lo;
      auto turn = [&](int i, auto buf) __attribute__((always_inline)) {
        constexpr int BUF = decltype(buf)::value, BEFORE = (BUF + RING - 1) % RING, NEXT = (BUF + 1) % RING;
        landed();
        __syncthreads();  // tile i and the probabilities of tile i - 1 are there; nobody reads tile i - 2 any more
        if (i + 1 < turns) {
          if (++ahead == t_hi) ahead = t_lo, ++ahead_hd;
          fetch(ahead_hd, ahead, NEXT);
        }
        if (careful && i < turns && hides((t_lo + i % nt) * QT)) {
          // (lse and delta of a row hold what its odd values made of it)
          clean<BF16, TILE>(sm.tile[BUF][0], tid);
          clean<BF16, TILE>(sm.tile[BUF][1], tid);
        }
        if constexpr (SECOND) {
          if (i == 0) return;
          if (hides(t * QT)) slopes(t * QT, BEFORE, std::true_type{});
          else slopes(t * QT, BEFORE, std::false_type{});
        } else {
          if (i == turns) return;
          if (hides(t * QT)) scores(t * QT, BUF, std::true_type{});
          else scores(t * QT, BUF, std::false_type{});
        }
        if (++t == t_hi) t = t_lo;
      };
      for (int i = 0; i <= turns; i += RING) {
        turn(i, std::integral_constant<int, 0>{});
        if (i + 1 <= turns) turn(i + 1, std::integral_constant<int, 1>{});
        if (i + 2 <= turns) turn(i + 2, std::integral_constant<int, 2>{});
      }
    };
    if (second) walk(std::true_type{});
    else walk(std::false_type{});
    if (careful) {
#pragma unroll 1
      for (int i = 0; i < turns; ++i) {
        const int q0 = (t_lo + i % nt) * QT;
        if (!hides(q0)) continue;
        __syncthreads();
        fetch(i / nt, t_lo + i % nt, 0);
        landed();
        __syncthreads();
        if (second) restore<BF16, D, QT, false>(acc, sm.tile[0][0], first - q0, last - q0, h);
        else restore<BF16, D, QT, true>(acc, sm.tile[0][1], first - q0, last - q0, h);
      }
      break;
    }
    if (!any_wave(any_odd(acc), sm.said, tid)) break;
  }
  if (mine >= m.nk) return;
  const float f = !second ? 1.f : all_lone ? 0.f : p.scale;
  const int64_t to = ((sp.k0 + mine) * (int64_t)p.Hkv + kv) * D;
  if (p.parts == 1) {
    store_row<BF16, D>(static_cast<char *>(second ? p.dk : p.dv) + to * ES, acc, f, h);
  } else {
    const int64_t n = (int64_t)(p.cu_q ? 1 : p.B) * p.Tk * p.Hkv * D;
    store_row<false, D>(reinterpret_cast<char *>(p.partial + (2 * slice + !second) * n + to), acc, f, h);
  }
}

// Sums of the parts, in order; four values a thread. Rows of no sequence: see the next kernel.
template <bool BF16> __global__ void __launch_bounds__(256) attention_join_kernel(const AttentionArgs p, int64_t n) {
  const int64_t w = (int64_t)p.Hkv * p.d, from = p.cu_q ? clamp_to(p.cu_k[0], p.Tk) * w : 0;
  const int64_t to = p.cu_q ? clamp_to(p.cu_k[p.B], p.Tk) * w : n;
  for (int64_t i = from + 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < to; i += 1024 * (int64_t)gridDim.x)
    for (int out = 0; out < 2; ++out) {
      floatx4 x = *reinterpret_cast<const floatx4 *>(p.partial + out * n + i);
      for (int k = 1; k < p.parts; ++k) x += *reinterpret_cast<const floatx4 *>(p.partial + (2 * k + out) * n + i);
      const float y[4] = {x[0], x[1], x[2], x[3]};
      store_f<BF16, 4>(out ? p.dv : p.dk, (size_t)i, y);
    }
}

// Gradients of packed tokens of no sequence: zero. One workgroup row by row of the tokens before the first and
// behind the last sequence.
__global__ void __launch_bounds__(256) attention_outside_kernel(const AttentionArgs p, int es) {
  for (int side = 0; side < 2; ++side) {
    const int32_t *cu = side ? p.cu_k : p.cu_q;
    const int T = side ? p.Tk : p.Tq, a = p.B ? clamp_to(cu[0], T) : 0, b = p.B ? max(clamp_to(cu[p.B], T), a) : 0;
    const int64_t w = (int64_t)(side ? p.Hkv : p.H) * p.d * es / 16;  // 16-byte pieces of a row
    const int64_t n = ((int64_t)a + T - b) * w;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
      const int64_t at = i < a * w ? i : i + (b - a) * w;
      const uintx4 z = {0, 0, 0, 0};
      if (side) {
        reinterpret_cast<uintx4 *>(p.dk)[at] = z;
        reinterpret_cast<uintx4 *>(p.dv)[at] = z;
      } else {
        reinterpret_cast<uintx4 *>(p.dq)[at] = z;
      }
    }
  }
}

template <bool BF16, int D> hipError_t run(const AttentionArgs &p, hipStream_t stream) {
  const bool packed = p.cu_q != nullptr;
  const size_t seqs = packed ? 1 : (size_t)p.B;
  auto tiles = [&](int rows) { return attention_blocks(packed ? p.B : 1, p.Tq, rows, packed); };
  const size_t uq = seqs * (size_t)p.H;
  if (tiles(kAttnRows)) {
    // as in the forward
    const size_t enough = (!BF16 && D == 128) || p.window || !p.causal ? 256 : 512;
    if (tiles(kAttnRows) * uq <= enough)
      attention_dq_kernel<BF16, D, 2><<<(unsigned)(tiles(kAttnRows / 2) * uq), 256, 0, stream>>>(p, (unsigned)uq);
    else
      attention_dq_kernel<BF16, D, 1><<<(unsigned)(tiles(kAttnRows) * uq), 256, 0, stream>>>(p, (unsigned)uq);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const size_t tk = attention_blocks(packed ? p.B : 1, p.Tk, p.keys, packed), uk = seqs * (size_t)p.Hkv * (size_t)p.parts;
  if (!tk) return hipSuccess;
  // fp32 at d 128 has 128 keys alone: two workgroups of 64 do not fit a CU's LDS
  if (p.keys == 64 && (BF16 || D == 64))
    attention_dkv_kernel<BF16, D, BF16 || D == 64 ? 64 : 128><<<(unsigned)(tk * uk), 256, 0, stream>>>(p, (unsigned)uk);
  else
    attention_dkv_kernel<BF16, D, 128><<<(unsigned)(tk * uk), 512, 0, stream>>>(p, (unsigned)uk);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (p.parts > 1) {
    const int64_t n = (int64_t)seqs * p.Tk * p.Hkv * D;
    const int64_t groups = (n / 4 + 255) / 256;
    attention_join_kernel<BF16><<<(unsigned)(groups < 65536 ? groups : 65536), 256, 0, stream>>>(p, n);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Keys: 64 a workgroup, two of which share a CU and do not wait for each other, where d is 64 (B4 T4096 H32/4 bf16:
// backward 1143 us, 1220 with 128), under a window (T4096 window 512 H16/2 d128: 707 against 793) and where 128 would
// leave CUs without any; else 128, whose queries cross LDS once for twice as many keys (B4 T4096 H16/2 d128: 1025
// against 1059).
// Parts: a key block's workgroup walks the query heads that share it. Where there are few such blocks the heads are
// dealt out to several workgroups, whose sums are joined in order: 1024 of 128 keys, or 2048 of 64, even out blocks
// that are seen by many queries and by few (the d 64 shape above with 1024 of 64: 1217 us); under a window, where all
// are seen alike, 512 are enough (the shape above with 2048 of 64: 744 us).
AttentionSplit attention_backward_split(int B, int Tk, int H, int Hkv, int d, bool bf16, int window, bool packed) {
  auto blocks = [&](int keys) {
    return (packed ? (size_t)Tk / keys + 1 : attention_blocks(1, Tk, keys, false) * (size_t)B) * (size_t)Hkv;
  };
  const int group = H / Hkv;
  AttentionSplit s;
  s.keys = (bf16 || d == 64) && (d == 64 || window || blocks(128) * group < 256) ? 64 : 128;
  const size_t enough = window ? 512 : s.keys == 64 ? 2048 : 1024;
  for (s.parts = 1; s.parts < group; ++s.parts)
    if (group % s.parts == 0 && blocks(s.keys) * s.parts >= enough) break;
  return s;
}

hipError_t launch_attention_backward(const AttentionArgs &p, hipStream_t stream) {
  if (p.cu_q) {
    attention_outside_kernel<<<256, 256, 0, stream>>>(p, p.bf16 ? 2 : 4);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!p.B) return hipSuccess;
  if (p.bf16) return p.d == 128 ? run<true, 128>(p, stream) : run<true, 64>(p, stream);
  return p.d == 128 ? run<false, 128>(p, stream) : run<false, 64>(p, stream);
}

}  // namespace gdn2
