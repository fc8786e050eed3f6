// gdn2_attention.hip -- softmax attention over whole sequences, forward.
//
// o_i = sum_j p_ij v_j, p_ij = exp(s_ij - lse_i), s_ij = scale q_i . k_j over
// the keys j that query i sees. A workgroup takes 128 queries of one head, a
// wave 32 of them, and walks the keys in tiles that LDS holds twice, the next
// one on its way from memory. Scores are computed transposed (keys as
// rows), so that a query's softmax is a sum over its lane's registers and the
// probabilities are the next product's operand where they lie.
#include "gdn2_attention_device.hpp"

namespace gdn2 {
namespace {

using namespace attn;

// The running maximum follows a tile's only where it grows by more than this
// (powers of two): a sum of terms up to 2^8 is as exact in fp32 as one of terms
// up to 1, and so are bf16 probabilities; the rescaling of the accumulator is
// left out for nearly every tile.
constexpr float kSlack = 8.f;

template <bool BF16, int D> struct Forward {
  static constexpr int KT = BF16 ? 64 : 32;  // keys of a tile: 16 KB of each of K and V at D = 128
  using L = Tile<BF16, D>;
  static constexpr int TILE = KT * L::ROW;
};

template <bool BF16, int D>
__global__ void __launch_bounds__(256, BF16 || D == 64 ? 2 : 1) attention_forward_kernel(const AttentionArgs p, unsigned total, unsigned tiles) {
  using C = Forward<BF16, D>;
  using L = typename C::L;
  constexpr int KT = C::KT, SUB = KT / 32, ES = BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[2][2][C::TILE];  // first: within the 64 KB that m0 addresses
    Odd<BF16, D, KT> notes;
  } sm;
  unsigned unit, tile;
  if (!find_work(total, tiles, &unit, &tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int seq, row0, head;
  if (p.cu_q) {
    if (!find_block(p.cu_q, p.B, p.Tq, (int)tile, &seq, &row0)) return;
    head = (int)unit;
  } else {
    seq = (int)(unit / (unsigned)p.H);
    head = (int)(unit % (unsigned)p.H);
    row0 = (int)tile * kAttnRows;
  }
  const Span sp = span_of(p, seq, head);
  const Mask m = sp.m;
  if (row0 >= m.nq) return;
  const int kv = head / (p.H / p.Hkv);
  const char *kbase = static_cast<const char *>(p.k) + (sp.k0 * p.sk + (int64_t)kv * D) * ES;
  const char *vbase = static_cast<const char *>(p.v) + (sp.k0 * p.sv + (int64_t)kv * D) * ES;

  // this lane's query, and the rows of its wave
  const int wrow = row0 + 32 * wave, mine = wrow + (lane & 31), row = min(mine, m.nq - 1);
  const int wlast = min(wrow + 31, m.nq - 1);  // < wrow: a wave without queries
  Frag<BF16> q[D / 16];
  load_row<BF16, D>(q, static_cast<const char *>(p.q) + ((sp.q0 + row) * p.sq + (int64_t)head * D) * ES, h);
  arrived(q);
  const float c = p.scale * kLog2e;
  const int hi = m.hi(row), lo = m.lo(row);
  // tiles that some query of the workgroup, and of the wave, sees; keys that
  // every query of the workgroup, and of the wave, sees
  const int blast = min(row0 + kAttnRows - 1, m.nq - 1);
  const int t_lo = m.lo(row0) / KT, t_hi = (m.hi(blast) + KT) / KT;  // hi = -1: none
  const int w_lo = m.lo(min(wrow, m.nq - 1)), w_hi = wrow <= wlast ? m.hi(wlast) : -1;
  const int b_lo = m.lo(blast), b_hi = m.hi(row0);
  const int all_lo = m.lo(max(wlast, 0)), all_hi = m.hi(min(wrow, m.nq - 1));

  floatx16 acc[D / 32];
#pragma unroll
  for (int b = 0; b < D / 32; ++b) acc[b] = zero16();
  float top = neg_inf(), sum = 0.f;

  // One tile's products. masked (uniform): some query does not see some key.
  auto step = [&](const char *kt, const char *vt, int key0, bool masked) __attribute__((always_inline)) {
    floatx16 s[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) s[u] = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int u = 0; u < SUB; ++u) s[u] = mma<BF16>(s[u], L::along(kt, 32 * u + (lane & 31), kk, h), q[kk]);
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
    t = other_half_max(t) * c;
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
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], c, -base));
        sum += s[u][i];
      }
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // bf16: the probabilities' one rounding, 2^-9 of each at most
        const Frag<BF16> w = operand<BF16>(s[u], g);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) acc[b] = mma<BF16>(acc[b], L::across(vt, 32 * u + 16 * g, 32 * b, lane), w);
      }
  };

  if (t_lo < t_hi) {
    Dma<BF16, D, KT> ks, vs;
    ks.init(p.sk * ES, tid);
    vs.init(p.sv * ES, tid);
    ks.load(sm.tile[0][0], kbase, t_lo * KT, m.nk, wave);
    vs.load(sm.tile[0][1], vbase, t_lo * KT, m.nk, wave);
    // BUF: the tile's buffer, a constant, so that LDS addresses are a lane's own and an offset
    auto turn = [&](int t, auto buf) __attribute__((always_inline)) {
      constexpr int BUF = decltype(buf)::value;
      const int key0 = t * KT;
      landed();
      __syncthreads();  // tile t is there, and nobody reads tile t - 1 any more
      if (t + 1 < t_hi) {
        ks.load(sm.tile[BUF ^ 1][0], kbase, key0 + KT, m.nk, wave);
        vs.load(sm.tile[BUF ^ 1][1], vbase, key0 + KT, m.nk, wave);
      }
      char *kt = sm.tile[BUF][0], *vt = sm.tile[BUF][1];
      const bool bad = (key0 < b_lo || key0 + KT - 1 > b_hi) && clean<BF16, D, KT>(vt, sm.notes, tid);
      if (key0 <= w_hi && key0 + KT > w_lo) step(kt, vt, key0, key0 < all_lo || key0 + KT - 1 > all_hi);
      if (bad) poison<BF16, D, KT>(acc, sm.notes, lo - key0, hi - key0, h);
    };
    for (int t = t_lo; t < t_hi; t += 2) {
      turn(t, std::integral_constant<int, 0>{});
      if (t + 1 < t_hi) turn(t + 1, std::integral_constant<int, 1>{});
    }
  }

  if (mine >= m.nq) return;
  sum = other_half_sum(sum);
  const bool empty = hi < lo;  // no key at all: zero, and a log-sum of -inf
  char *out = static_cast<char *>(p.o) + ((sp.q0 + mine) * (int64_t)p.H + head) * D * ES;
  store_row<BF16, D>(out, acc, empty ? 0.f : 1.f / sum, h);
  if (h == 0 && p.lse) p.lse[sp.rows + mine] = empty ? neg_inf() : __builtin_fmaf(top, kLn2, __logf(sum));
}

template <bool BF16, int D> hipError_t run(const AttentionArgs &p, hipStream_t stream) {
  const size_t tiles = attention_tiles(p.cu_q ? p.B : 1, p.Tq, p.cu_q != nullptr);
  const size_t total = tiles * (p.cu_q ? 1 : (size_t)p.B) * (size_t)p.H;
  if (!total) return hipSuccess;
  const unsigned grid = (unsigned)((total + 7) / 8 * 8);
  attention_forward_kernel<BF16, D><<<grid, 256, 0, stream>>>(p, (unsigned)total, (unsigned)tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_forward(const AttentionArgs &p, hipStream_t stream) {
  if (p.bf16) return p.d == 128 ? run<true, 128>(p, stream) : run<true, 64>(p, stream);
  return p.d == 128 ? run<false, 128>(p, stream) : run<false, 64>(p, stream);
}

}  // namespace gdn2
