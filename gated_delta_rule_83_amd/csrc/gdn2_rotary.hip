// gdn2_rotary.hip -- queries' and keys' root-mean-square norm for each head and
// their rotation by position, in one pass, and its gradients.
//
//   u = x / sqrt(mean(x^2) + eps) * w      (u_a, u_b) -> (u_a c - u_b s, u_b c + u_a s)
//
// with c, s the cosine and sine of position * inv_freq[pair]. HBM bounds it:
// every row is read once and written once. A lane holds two pieces of 4 values
// whose pairs it has whole, a row lies on 2 to 32 lanes of a wave, so a wave has
// several heads of one token at once; its 64 lanes compute the token's sines
// once for all of its heads. The angle is a product of 55 bits, times 1 / (2 pi):
// both products keep what their rounding to 64 bits leaves, so that a turn's
// fraction is as exact at position 2^31 as at 1 (without, up to 4e-7 of a radian
// off there); then it is rounded to fp32.
#include "gdn2_rotary.hpp"
#include "gdn2_vec.hpp"

namespace gdn2 {
namespace {

constexpr int kWaves = 4;

__device__ __forceinline__ void turn_of(int position, float inv_freq, float *c, float *s) {
  constexpr double kTurn = 0.15915494309189533577, kTurnLow = -9.839338337591243e-18;  // 1 / (2 pi), and the rest of it
  const double p = position, f = inv_freq, a = p * f, low = __builtin_fma(p, f, -a);  // p f = a + low
  const double part = __builtin_fma(a, kTurn, -__builtin_rint(a * kTurn));
  const float x = (float)(2.0 * (part + __builtin_fma(a, kTurnLow, low * kTurn)));  // half turns, -1 .. 1
  sincospif(x, s, c);
}

// How rows lie on lanes. WIDE: LANES lanes a row, 4 pairs each, wide loads (d and rot multiples of 8, all
// aligned). Otherwise a wave a row and single values, up to 8 pairs a lane.
template <bool WIDE_, int LANES_> struct Plan {
  static constexpr bool WIDE = WIDE_;
  static constexpr int LANES = LANES_, ROWS = 64 / LANES, PAIRS = WIDE ? 4 : kRotaryMaxD / 128;
};

template <class P, bool BF16, bool NEIGHBOURS> struct Row {
  static constexpr int N = P::PAIRS, ES = BF16 ? 2 : 4;
  float a[N], b[N];  // the two values of each pair

  // values of pair j of lane l, and whether there are any
  static __device__ __forceinline__ bool places(int l, int j, int d, int rot, int *ea, int *eb) {
    const int p = l + 64 * j, half = rot / 2;
    const bool turned = p < half;
    *ea = turned && !NEIGHBOURS ? p : 2 * p - (turned ? 0 : rot - 2 * half);
    if (!turned) *ea = rot + 2 * (p - half);
    *eb = turned && !NEIGHBOURS ? p + half : *ea + 1;
    return p < d / 2;
  }
  // the wide plan's pieces
  static __device__ __forceinline__ void pieces(int l, int rot, int *oa, int *ob) {
    const bool halves = !NEIGHBOURS && 8 * l < rot;
    *oa = halves ? 4 * l : 8 * l;
    *ob = halves ? rot / 2 + 4 * l : 8 * l + 4;
  }
  template <bool B> __device__ __forceinline__ void load(const char *row, int l, int d, int rot) {
    constexpr int E = B ? 2 : 4;
    if constexpr (P::WIDE) {
      int oa, ob;
      pieces(l, rot, &oa, &ob);
      float x[4] = {}, y[4] = {};
      if (8 * l < d) {
        load_f<B, 4>(x, row + oa * E, 0);
        load_f<B, 4>(y, row + ob * E, 0);
      }
      sort(x, y);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        int ea, eb;
        const bool have = places(l, j, d, rot, &ea, &eb);
        using T = typename Elem<B>::T;
        a[j] = have ? Elem<B>::ld(reinterpret_cast<const T *>(row) + ea) : 0.f;
        b[j] = have ? Elem<B>::ld(reinterpret_cast<const T *>(row) + eb) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void sort(const float (&x)[4], const float (&y)[4]) {
    if constexpr (NEIGHBOURS) {
      a[0] = x[0], b[0] = x[1], a[1] = x[2], b[1] = x[3], a[2] = y[0], b[2] = y[1], a[3] = y[2], b[3] = y[3];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = x[j], b[j] = y[j];
    }
  }
  template <bool B> __device__ __forceinline__ void store(char *row, int l, int d, int rot) const {
    constexpr int E = B ? 2 : 4;
    if constexpr (P::WIDE) {
      if (8 * l >= d) return;
      int oa, ob;
      pieces(l, rot, &oa, &ob);
      float x[4], y[4];
      if constexpr (NEIGHBOURS) {
        x[0] = a[0], x[1] = b[0], x[2] = a[1], x[3] = b[1], y[0] = a[2], y[1] = b[2], y[2] = a[3], y[3] = b[3];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = a[j], y[j] = b[j];
      }
      store_at<B, 4>(row + oa * E, x);
      store_at<B, 4>(row + ob * E, y);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        int ea, eb;
        if (!places(l, j, d, rot, &ea, &eb)) continue;
        using T = typename Elem<B>::T;
        Elem<B>::st(reinterpret_cast<T *>(row) + ea, a[j]);
        Elem<B>::st(reinterpret_cast<T *>(row) + eb, b[j]);
      }
    }
  }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = b[j] = x;
  }
  __device__ __forceinline__ void times(const Row &o) {
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] *= o.a[j], b[j] *= o.b[j];
  }
  // the sum of o's products with this row, over the row's lanes
  __device__ __forceinline__ float dot(const Row &o) const {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) s = __builtin_fmaf(a[j], o.a[j], __builtin_fmaf(b[j], o.b[j], s));
    return lane_sum<P::LANES>(s);
  }
};

// Cosines and sines of this lane's pairs.
template <class P> struct Turn {
  float c[P::PAIRS], s[P::PAIRS];
  // share: this wave's 2 x 128 values in LDS (wide plans)
  __device__ __forceinline__ void set(int position, const float *inv_freq, int rot, int lane, float *share) {
    const int half = rot / 2;
    if constexpr (P::WIDE) {
      constexpr int MOST = P::LANES * 4;  // pairs of a row
#pragma unroll
      for (int i = 0; i < (MOST + 63) / 64; ++i) {
        const int pair = lane + 64 * i;
        if (pair < MOST) {
          float cc = 1.f, ss = 0.f;
          if (pair < half) turn_of(position, inv_freq[pair], &cc, &ss);
          share[pair] = cc;
          share[128 + pair] = ss;
        }
      }
      __builtin_amdgcn_wave_barrier();
      const int l = lane % P::LANES;
      const floatx4 cv = *reinterpret_cast<const floatx4 *>(share + 4 * l), sv = *reinterpret_cast<const floatx4 *>(share + 128 + 4 * l);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = cv[j], s[j] = sv[j];
      __builtin_amdgcn_wave_barrier();
    } else {
#pragma unroll
      for (int j = 0; j < P::PAIRS; ++j) {
        c[j] = 1.f, s[j] = 0.f;
        if (lane + 64 * j < half) turn_of(position, inv_freq[lane + 64 * j], &c[j], &s[j]);
      }
    }
  }
};

// Work: (token, piece of its heads) in turn over the waves of the grid.
template <class P, bool BF16, bool WBF16, bool NEIGHBOURS>
__global__ void __launch_bounds__(256) rotary_forward_kernel(const RotaryArgs p, int pieces, int heads) {
  using R = Row<P, BF16, NEIGHBOURS>;
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ float share[P::WIDE ? kWaves : 1][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % P::LANES, sub = lane / P::LANES;
  R qw, kw;
  qw.fill(1.f);
  kw.fill(1.f);
  if (p.qw) qw.template load<WBF16>(static_cast<const char *>(p.qw), l, p.d, p.rot);
  if (p.kw) kw.template load<WBF16>(static_cast<const char *>(p.kw), l, p.d, p.rot);
  const int all = p.Hq + p.Hk;
  const int64_t work = p.tokens * pieces;
  for (int64_t w = (int64_t)blockIdx.x * kWaves + wave; w < work; w += (int64_t)gridDim.x * kWaves) {
    const int64_t token = pieces == 1 ? w : w / pieces;
    const int first = pieces == 1 ? 0 : (int)(w % pieces) * heads, end = min(first + heads, all);
    Turn<P> turn;
    turn.set(p.positions[token], p.inv_freq, p.rot, lane, share[P::WIDE ? wave : 0]);
    const char *q = static_cast<const char *>(p.q) + token * p.sq * ES, *k = static_cast<const char *>(p.k) + token * p.sk * ES;
    for (int h0 = first; h0 < end; h0 += P::ROWS) {
      const int h = h0 + sub;
      const bool live = h < end, key = h >= p.Hq;
      const int64_t at = (int64_t)(key ? h - p.Hq : h) * p.d * ES;
      R x;
      if (live) x.template load<BF16>((key ? k : q) + at, l, p.d, p.rot);
      else x.fill(0.f);
      float r = 1.f;
      if (p.norm) r = 1.f / __builtin_sqrtf(x.dot(x) / (float)p.d + p.eps);
      R y;
#pragma unroll
      for (int j = 0; j < P::PAIRS; ++j) {
        const float a = x.a[j] * r * (key ? kw.a[j] : qw.a[j]), b = x.b[j] * r * (key ? kw.b[j] : qw.b[j]);
        y.a[j] = a * turn.c[j] - b * turn.s[j];
        y.b[j] = b * turn.c[j] + a * turn.s[j];
      }
      if (live)
        y.template store<BF16>((key ? static_cast<char *>(p.k_out) + token * p.Hk * p.d * ES
                                    : static_cast<char *>(p.q_out) + token * p.Hq * p.d * ES) + at, l, p.d, p.rot);
    }
  }
}

//   du = dy turned back,  dw = sum du xh,  dx = r (du w - xh mean(du w xh))
// The weights' sums stay in registers over all of a wave's rows; then one row
// of [2][d] a workgroup, which the next kernel adds up in a fixed order.
template <class P, bool BF16, bool WBF16, bool NEIGHBOURS>
__global__ void __launch_bounds__(256, P::WIDE ? 5 : 2) rotary_backward_kernel(const RotaryArgs p, int pieces, int heads) {
  using R = Row<P, BF16, NEIGHBOURS>;
  constexpr int ES = BF16 ? 2 : 4;
  __shared__ float share[P::WIDE ? kWaves : 1][256];
  extern __shared__ float sums[];  // [kWaves][2][d], where weights' gradients are wanted
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % P::LANES, sub = lane / P::LANES;
  R qw, kw, dqw, dkw;
  qw.fill(1.f);
  kw.fill(1.f);
  dqw.fill(0.f);
  dkw.fill(0.f);
  if (p.qw) qw.template load<WBF16>(static_cast<const char *>(p.qw), l, p.d, p.rot);
  if (p.kw) kw.template load<WBF16>(static_cast<const char *>(p.kw), l, p.d, p.rot);
  const int all = p.Hq + p.Hk;
  const int64_t work = p.tokens * pieces;
  for (int64_t w = (int64_t)blockIdx.x * kWaves + wave; w < work; w += (int64_t)gridDim.x * kWaves) {
    const int64_t token = pieces == 1 ? w : w / pieces;
    const int first = pieces == 1 ? 0 : (int)(w % pieces) * heads, end = min(first + heads, all);
    Turn<P> turn;
    turn.set(p.positions[token], p.inv_freq, p.rot, lane, share[P::WIDE ? wave : 0]);
    const char *q = static_cast<const char *>(p.q) + token * p.sq * ES, *k = static_cast<const char *>(p.k) + token * p.sk * ES;
    const int64_t qat = token * p.Hq * p.d * ES, kat = token * p.Hk * p.d * ES;
    for (int h0 = first; h0 < end; h0 += P::ROWS) {
      const int h = h0 + sub;
      const bool live = h < end, key = h >= p.Hq;
      const int64_t at = (int64_t)(key ? h - p.Hq : h) * p.d * ES, out = (key ? kat : qat) + at;
      R x, g;
      if (live) {
        x.template load<BF16>((key ? k : q) + at, l, p.d, p.rot);
        g.template load<BF16>(static_cast<const char *>(key ? p.gk : p.gq) + out, l, p.d, p.rot);
      } else {
        x.fill(0.f);
        g.fill(0.f);
      }
      float r = 1.f;
      if (p.norm) r = 1.f / __builtin_sqrtf(x.dot(x) / (float)p.d + p.eps);
      r = live ? r : 0.f;  // lanes without a head: 1 / 0 where eps is, and NaN times zero in a weight's sum
#pragma unroll
      for (int j = 0; j < P::PAIRS; ++j) {
        const float a = g.a[j] * turn.c[j] + g.b[j] * turn.s[j], b = g.b[j] * turn.c[j] - g.a[j] * turn.s[j];
        x.a[j] *= r, x.b[j] *= r;
        const float wa = a * x.a[j], wb = b * x.b[j];
        if (key) dkw.a[j] += wa, dkw.b[j] += wb;
        else dqw.a[j] += wa, dqw.b[j] += wb;
        g.a[j] = a * (key ? kw.a[j] : qw.a[j]);
        g.b[j] = b * (key ? kw.b[j] : qw.b[j]);
      }
      const float m = p.norm ? g.dot(x) / (float)p.d : 0.f;
#pragma unroll
      for (int j = 0; j < P::PAIRS; ++j) g.a[j] = r * (g.a[j] - x.a[j] * m), g.b[j] = r * (g.b[j] - x.b[j] * m);
      if (live) g.template store<BF16>(static_cast<char *>(key ? p.dk : p.dq) + out, l, p.d, p.rot);
    }
  }
  if (!p.dqw && !p.dkw) return;
  // lanes of the same place of a row, then the waves
#pragma unroll
  for (int x = P::LANES; x < 64; x <<= 1)
#pragma unroll
    for (int j = 0; j < P::PAIRS; ++j) {
      dqw.a[j] += __shfl_xor(dqw.a[j], x), dqw.b[j] += __shfl_xor(dqw.b[j], x);
      dkw.a[j] += __shfl_xor(dkw.a[j], x), dkw.b[j] += __shfl_xor(dkw.b[j], x);
    }
  if (sub == 0) {
    dqw.template store<false>(reinterpret_cast<char *>(sums + (2 * wave) * p.d), l, p.d, p.rot);
    dkw.template store<false>(reinterpret_cast<char *>(sums + (2 * wave + 1) * p.d), l, p.d, p.rot);
  }
  __syncthreads();
  float *to = static_cast<float *>(p.workspace) + (int64_t)blockIdx.x * 2 * p.d;
  for (int i = threadIdx.x; i < 2 * p.d; i += 256) to[i] = sums[i] + sums[2 * p.d + i] + sums[4 * p.d + i] + sums[6 * p.d + i];
}

// [rows][2 d] partial sums to dqw and dkw: 16 columns a workgroup, 16 threads a column.
template <bool WBF16> __global__ void __launch_bounds__(256) rotary_weight_kernel(const RotaryArgs p, int rows) {
  __shared__ float part[16][17];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4, col = blockIdx.x * 16 + c;
  float s = 0.f;
  if (col < 2 * p.d) {
    const float *from = static_cast<const float *>(p.workspace) + col;
#pragma unroll 4
    for (int r = g; r < rows; r += 16) s += from[(int64_t)r * 2 * p.d];
  }
  part[g][c] = s;
  __syncthreads();
  if (g || col >= 2 * p.d) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += part[i][c];
  void *out = col < p.d ? p.dqw : p.dkw;
  const float y[1] = {s};
  if (out) store_f<WBF16, 1>(out, (size_t)(col % p.d), y);
}

struct Grid {
  int pieces, heads;
  unsigned groups;
};
// A wave takes a token's heads one after another, so that its sines serve all of
// them; where that leaves fewer than 8 waves a CU the heads are dealt out too.
Grid grid_of(int64_t tokens, int all, int rows, unsigned most) {
  if (tokens == 0) return Grid{1, all, 0};
  Grid g;
  const int steps = (all + rows - 1) / rows;
  int64_t pieces = tokens >= 2048 ? 1 : (2048 + tokens - 1) / tokens;
  if (pieces > steps) pieces = steps;
  const int per = (int)((steps + pieces - 1) / pieces);
  g.heads = per * rows;
  g.pieces = (steps + per - 1) / per;
  const int64_t groups = (tokens * g.pieces + kWaves - 1) / kWaves;
  g.groups = (unsigned)(groups < most ? groups : most);
  return g;
}

// Forward: more workgroups than fit, so that the card's dies end together (32768 tokens H16/2 d128 bf16: 56 us, 65 with
// 2048). Backward: as many as fit, 5 a CU by its registers, whose weights' sums are one row each (102 us; 113 with
// 1024, 119 with 2048).
constexpr unsigned kForwardGroups = 8192, kBackwardGroups = 1280;

bool wide(const RotaryArgs &p, bool backward) {
  const uintptr_t es = p.bf16 ? 2 : 4, ws = p.wbf16 ? 2 : 4;
  // 4 values at a time; 16 bytes is the widest of them
  auto ok = [](const void *x, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(x) & (4 * bytes - 1)) == 0; };
  bool a = p.d % 8 == 0 && p.rot % 8 == 0 && p.d <= 256 && p.sq % 4 == 0 && p.sk % 4 == 0;
  a = a && ok(p.q, es) && ok(p.k, es) && ok(p.qw, ws) && ok(p.kw, ws);
  if (backward) return a && ok(p.gq, es) && ok(p.gk, es) && ok(p.dq, es) && ok(p.dk, es);
  return a && ok(p.q_out, es) && ok(p.k_out, es);
}

template <class P, bool BF16, bool WBF16, bool NEIGHBOURS>
hipError_t run(const RotaryArgs &p, bool backward, hipStream_t stream) {
  const Grid g = grid_of(p.tokens, p.Hq + p.Hk, P::ROWS, backward ? kBackwardGroups : kForwardGroups);
  if (!backward) {
    rotary_forward_kernel<P, BF16, WBF16, NEIGHBOURS><<<g.groups, 256, 0, stream>>>(p, g.pieces, g.heads);
    return hipGetLastError();
  }
  const bool weights = p.dqw || p.dkw;
  if (g.groups) {
    rotary_backward_kernel<P, BF16, WBF16, NEIGHBOURS>
        <<<g.groups, 256, weights ? kWaves * 2 * p.d * 4 : 0, stream>>>(p, g.pieces, g.heads);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (weights) {
    rotary_weight_kernel<WBF16><<<(unsigned)(2 * p.d + 15) / 16, 256, 0, stream>>>(p, (int)g.groups);
    return hipGetLastError();
  }
  return hipSuccess;
}

template <bool BF16, bool WBF16, bool NEIGHBOURS> hipError_t by_width(const RotaryArgs &p, bool backward, hipStream_t stream) {
  if (!wide(p, backward)) return run<Plan<false, 64>, BF16, WBF16, NEIGHBOURS>(p, backward, stream);
  if (p.d <= 32) return run<Plan<true, 4>, BF16, WBF16, NEIGHBOURS>(p, backward, stream);
  if (p.d <= 64) return run<Plan<true, 8>, BF16, WBF16, NEIGHBOURS>(p, backward, stream);
  if (p.d <= 128) return run<Plan<true, 16>, BF16, WBF16, NEIGHBOURS>(p, backward, stream);
  return run<Plan<true, 32>, BF16, WBF16, NEIGHBOURS>(p, backward, stream);
}

hipError_t launch(const RotaryArgs &p, bool backward, hipStream_t stream) {
  if (p.neighbours) {
    if (p.bf16) return p.wbf16 ? by_width<true, true, true>(p, backward, stream) : by_width<true, false, true>(p, backward, stream);
    return p.wbf16 ? by_width<false, true, true>(p, backward, stream) : by_width<false, false, true>(p, backward, stream);
  }
  if (p.bf16) return p.wbf16 ? by_width<true, true, false>(p, backward, stream) : by_width<true, false, false>(p, backward, stream);
  return p.wbf16 ? by_width<false, true, false>(p, backward, stream) : by_width<false, false, false>(p, backward, stream);
}

}  // namespace

size_t rotary_backward_workspace_bytes(int64_t tokens, int Hq, int Hk, int d) {
  // as many workgroups as any plan may have: at most 2048 waves more than there are tokens, or a wave a head
  const int64_t waves = tokens >= 2048 ? tokens : (2048 + tokens < tokens * (Hq + Hk) ? 2048 + tokens : tokens * (Hq + Hk));
  const int64_t groups = (waves + kWaves - 1) / kWaves;
  return (size_t)(groups < kBackwardGroups ? groups : kBackwardGroups) * 2 * (size_t)d * 4;
}

hipError_t launch_rotary_forward(const RotaryArgs &p, hipStream_t stream) { return launch(p, false, stream); }
hipError_t launch_rotary_backward(const RotaryArgs &p, hipStream_t stream) { return launch(p, true, stream); }

}  // namespace gdn2
