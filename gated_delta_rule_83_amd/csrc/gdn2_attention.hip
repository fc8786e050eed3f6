// gdn2_attention.hip -- softmax attention over whole sequences, forward.
//
// o_i = sum_j p_ij v_j, p_ij = exp(s_ij - lse_i), s_ij = scale q_i . k_j over
// the keys j that query i sees. A workgroup takes 128 queries of one head and
// walks the keys in tiles that LDS holds twice, the next one on its way from
// memory. Scores are computed transposed (keys as rows), so that a query's
// softmax is a sum over its lane's registers and the probabilities are the next
// product's operand where they lie.
#include "gdn2_attention_device.hpp"

namespace gdn2 {
namespace {

using namespace attn;

// The running maximum follows a tile's only where it grows by more than this
// (powers of two): a sum of terms up to 2^8 is as exact in fp32 as one of terms
// up to 1, and so are bf16 probabilities; the rescaling of the accumulator is
// left out for nearly every tile.
constexpr float kSlack = 8.f;

// SPLIT 2: 64 queries a workgroup; each 32 of them on two waves, which take half of
// every tile's keys each and join their sums in the end.
template <bool BF16, int D, int SPLIT>
__global__ void __launch_bounds__(256, BF16 || D == 64 ? 2 : 1) attention_forward_kernel(const AttentionArgs p, unsigned units) {
  using L = Tile<BF16, D>;
  constexpr int ROWS = kAttnRows / SPLIT, PAIRS = 4 / SPLIT;
  constexpr int KT = BF16 || SPLIT == 2 ? 64 : 32, SUB = KT / 32 / SPLIT, ES = BF16 ? 2 : 4;
  constexpr int TILE = KT * L::ROW;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[2][2][TILE];
    uint32_t said[4];
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

  // this lane's query, and the keys that it sees
  const int part = SPLIT == 1 ? 0 : wave / PAIRS, half = part * 32 * SUB;  // of the tiles' keys, from the half'th on
  const int mine = row0 + 32 * (wave % PAIRS) + (lane & 31), row = min(mine, m.nq - 1), hi = m.hi(row), lo = m.lo(row);
  Frag<BF16> q[D / 16];
  load_row<BF16, D>(q, static_cast<const char *>(p.q) + ((sp.q0 + row) * p.sq + (int64_t)head * D) * ES, h);
  arrived(q);
  const Exponent<BF16> power(p.scale);
  // tiles that some query of the workgroup sees; keys that every one of them sees
  const int blast = min(row0 + ROWS - 1, m.nq - 1);
  const int t_lo = m.lo(row0) / KT, t_hi = (m.hi(blast) + KT) / KT;  // hi = -1: none
  const int b_lo = m.lo(blast), b_hi = m.hi(row0);
  auto hides = [&](int key0) { return key0 < b_lo || key0 + KT - 1 > b_hi; };

  floatx16 acc[D / 32];
  float top, sum;
  Along<BF16, D> along;
  Across<BF16, D> across;
  along.init(lane, half);
  across.init(lane, half);
  const uint32_t at = lds_address(&sm);  // tile [i][j] from (2 i + j) TILE on
  Dma<BF16, D, KT> ks, vs;
  ks.init(p.sk * ES, tid);
  vs.init(p.sv * ES, tid);

  // scores of one tile: keys as rows
  auto scores = [&](floatx16 (&s)[SUB], uint32_t kt, int kk) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < SUB; ++u) s[u] = mma<BF16>(kk ? s[u] : zero16(), along.read(kt, 32 * u, kk), q[kk]);
  };
  // One tile from its scores `s`; meanwhile the next tile's scores, so that matrix
  // and vector instructions run side by side. masked (uniform): some query of the
  // workgroup does not see some key.
  auto step = [&](floatx16 (&s)[SUB], floatx16 (&next)[SUB], uint32_t vt, uint32_t next_kt, int key0,
                  bool masked) __attribute__((always_inline)) {
    if (masked) {
      // key key0 + 32 u + row_of(i, h) is seen where `from` <= 32 u + row_of(i, 0) <= `to`
      const int from = lo - key0 - 4 * h, to = hi - key0 - 4 * h;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * u + row_of(i, 0) < from || 32 * u + row_of(i, 0) > to) s[u][i] = neg_inf();
    }
    float t = neg_inf();
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) t = fmaxf(t, s[u][i]);
    t = other_half_max(t) * power.c;
    if (__any(t > top + kSlack)) {
      // each row by its own scores alone, whatever the wave's others do
      const bool grow = t > top + kSlack;
      const float f = grow ? __builtin_amdgcn_exp2f(top - t) : 1.f;
      top = grow ? t : top;
      sum *= f;
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] *= f;
    }
    const float base = top == neg_inf() ? 0.f : top;
    float own = 0.f;  // this tile's sum
    // Probabilities by groups of 8 registers, each the operand of one step of the
    // second product: the first half of them beside the next scores, each of the
    // others beside the product two (SUB) groups before it.
    auto weigh = [&](int group, int i) __attribute__((always_inline)) {
      floatx16 &x = s[group / 2];
      const int e = 8 * (group % 2) + i;
      x[e] = __builtin_amdgcn_exp2f(power(x[e], base));
      own += x[e];
    };
    constexpr int STEPS = D / 16, BLOCKS = D / 32;
    // the SIMD's other wave, in its own turn's vector part, lets the matrix products through
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < STEPS; ++kk) {
      scores(next, next_kt, kk);
#pragma unroll
      for (int i = kk * 8 * SUB / STEPS; i < (kk + 1) * 8 * SUB / STEPS; ++i) weigh(i / 8, i % 8);
    }
    if constexpr (BF16) {
#pragma unroll
      for (int g = 0; g < 2 * SUB; ++g) {
        // the probabilities' one rounding, 2^-8 of each at most
        const Frag<BF16> w = operand<BF16>(s[g / 2], g % 2);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
          acc[b] = mma<BF16>(acc[b], across.read(vt, 16 * g, b), w);
          if (g < SUB)
#pragma unroll
            for (int i = b * 8 / BLOCKS; i < (b + 1) * 8 / BLOCKS; ++i) weigh(g + SUB, i);
        }
      }
    } else {
      Frag<BF16> w[2 * SUB];
#pragma unroll
      for (int i = 8 * SUB; i < 16 * SUB; ++i) weigh(i / 8, i % 8);
#pragma unroll
      for (int g = 0; g < 2 * SUB; ++g) w[g] = operand<BF16>(s[g / 2], g % 2);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) add_products<BF16>(acc[b], [&](int g) { return across.read(vt, 16 * g, b); }, w);
    }
    sum += own;
    __builtin_amdgcn_s_setprio(0);
  };

  for (bool careful = false;; careful = true) {
    top = neg_inf();
    sum = 0.f;
#pragma unroll
    for (int b = 0; b < D / 32; ++b) acc[b] = zero16();
    if (t_lo >= t_hi) break;
    ks.load(sm.tile[0][0], kbase, t_lo * KT, m.nk, wave);
    vs.load(sm.tile[0][1], vbase, t_lo * KT, m.nk, wave);
    if (t_lo + 1 < t_hi) ks.load(sm.tile[1][0], kbase, (t_lo + 1) * KT, m.nk, wave);
    landed();
    __syncthreads();
    floatx16 s[2][SUB];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) scores(s[0], at, kk);
    // BUF: the tile's buffer, a constant, so that LDS addresses are a lane's own and an offset
    auto turn = [&](int t, auto buf) __attribute__((always_inline)) {
      constexpr int BUF = decltype(buf)::value;
      const int key0 = t * KT;
      landed();
      __syncthreads();  // V of tile t and K of tile t + 1 are there, and nobody reads those before them any more
      if (t + 1 < t_hi) vs.load(sm.tile[BUF ^ 1][1], vbase, key0 + KT, m.nk, wave);
      if (t + 2 < t_hi) ks.load(sm.tile[BUF][0], kbase, key0 + 2 * KT, m.nk, wave);
      const bool masked = hides(key0);
      if (careful && masked) clean<BF16, TILE>(sm.tile[BUF][1], tid);
      // (behind the last tile: scores of what the buffer holds, which nobody uses)
      step(s[BUF], s[BUF ^ 1], at + (2 * BUF + 1) * TILE, at + 2 * (BUF ^ 1) * TILE, key0 + half, masked);
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
        vs.load(sm.tile[0][1], vbase, t * KT, m.nk, wave);
        landed();
        __syncthreads();
        restore<BF16, D, KT, true>(acc, sm.tile[0][1], max(lo - t * KT, half), min(hi - t * KT, half + 32 * SUB - 1), h);
      }
      break;
    }
    if (!any_wave(any_odd(acc), sm.said, tid)) break;
  }

  sum = other_half_sum(sum);
  if constexpr (SPLIT == 2) {
    // the second half's maximum, sum and accumulator into the first's, through what was the tiles' memory
    floatx4 *to = reinterpret_cast<floatx4 *>(&sm) + (wave % PAIRS) * (D / 32 * 4 + 1) * 64 + lane;
    __syncthreads();
    if (part) {
#pragma unroll
      for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(4 * b + i) * 64] = floatx4{acc[b][4 * i], acc[b][4 * i + 1], acc[b][4 * i + 2], acc[b][4 * i + 3]};
      to[D / 32 * 4 * 64] = floatx4{top, sum, 0.f, 0.f};
    }
    __syncthreads();
    if (part) return;
    const floatx4 other = to[D / 32 * 4 * 64];
    const float most = fmaxf(top, other[0]);
    // a half that saw no number above -inf: its sums are zero or NaN
    const float f = top == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(top - most);
    const float g = other[0] == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(other[0] - most);
    top = most;
    sum = f * sum + g * other[1];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const floatx4 x = to[(b * 4 + i / 4) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][i + e] = f * acc[b][i + e] + g * x[e];
      }
  }
  if (mine >= m.nq) return;
  // no key at all, or scores of -inf alone: zero, and a log-sum of -inf
  const bool empty = sum == 0.f;
  char *out = static_cast<char *>(p.o) + ((sp.q0 + mine) * (int64_t)p.H + head) * D * ES;
  store_row<BF16, D>(out, acc, empty ? 0.f : 1.f / sum, h);
  if (h == 0 && p.lse) p.lse[sp.rows + mine] = empty ? neg_inf() : __builtin_fmaf(top, kLn2, __builtin_fmaf(top, kLn2Low, __logf(sum)));
}

template <bool BF16, int D> hipError_t run(const AttentionArgs &p, hipStream_t stream) {
  const bool packed = p.cu_q != nullptr;
  auto tiles = [&](int rows) { return attention_blocks(packed ? p.B : 1, p.Tq, rows, packed); };
  const size_t units = (packed ? 1 : (size_t)p.B) * (size_t)p.H;
  if (!tiles(kAttnRows) || !units) return hipSuccess;
  // Where blocks of 128 queries are no more than run at once, half as deep ones are done sooner (us, 128 queries / 64):
  // B1 T4096 H16/2 d128 bf16 103 / 88, B1 T2048 H8/2 46 / 32, in fp32 297 / 170, B1 T200 H8 d64 9.8 / 7.1. Where there
  // are more, keys cross LDS for twice as many queries (B2 T4096 H16/2 d128 156 / 174, B8 563 / 651). 512 run at once,
  // 256 of fp32 at d 128 (B2 T2048 H16/2 332 / 362); if all are equally deep, 512 fill the card already (B1 T4096
  // window 300 27.8 / 31.3).
  const size_t enough = (!BF16 && D == 128) || p.window || !p.causal ? 256 : 512;
  if (tiles(kAttnRows) * units <= enough)
    attention_forward_kernel<BF16, D, 2><<<(unsigned)(tiles(kAttnRows / 2) * units), 256, 0, stream>>>(p, (unsigned)units);
  else
    attention_forward_kernel<BF16, D, 1><<<(unsigned)(tiles(kAttnRows) * units), 256, 0, stream>>>(p, (unsigned)units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_forward(const AttentionArgs &p, hipStream_t stream) {
  if (p.bf16) return p.d == 128 ? run<true, 128>(p, stream) : run<true, 64>(p, stream);
  return p.d == 128 ? run<false, 128>(p, stream) : run<false, 64>(p, stream);
}

}  // namespace gdn2
