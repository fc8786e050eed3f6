// gdn2_norm.hip -- layer norm and root-mean-square norm over the last axis,
// optionally times silu(gate), and their gradients.
//
//   c = x - mean(x) (layer) or x,  r = 1 / sqrt(mean(c^2) + eps),  xh = c r,
//   n = xh w + bias,  y = n silu(z)  (or n without a gate z).
// With dn = dy silu(z) and d = dn w:
//   dx = r (d - xh mean(d xh) - mean(d))   (the last term for layer norm only)
//   dw = sum over rows of dn xh,  dbias = sum over rows of dn,
//   dz = dy n silu'(z),  silu'(z) = s (1 + z (1 - s)),  s = sigmoid(z).
// The mean is taken first and the squares of the centred values second, so
// that a large common offset costs no accuracy. All sums are fp32.
//
// Bound by HBM: a row is read once and kept in registers between its sums. A
// row belongs to LPR lanes of a wave (narrow rows) or to a whole workgroup,
// each lane with NC pieces of V values (one wide load each); workgroups stay
// and walk the rows, the next row's loads in flight during this row's sums,
// so that the weights, and the backward's sums of the weights' gradients, stay
// in registers too.
#include "gdn2_norm.hpp"

#include <initializer_list>

#include "gdn2_vec.hpp"

namespace gdn2 {

namespace {

__device__ __forceinline__ float load_w(const void *p, int i, bool bf16, float none) {
  if (!p) return none;
  return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_w(void *p, int i, bool bf16, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = f32_to_bf16(v);
  else
    static_cast<float *>(p)[i] = v;
}

// 1 / (1 + e^-z); z below -87 counts as -87 (2e-38), NaN stays.
__device__ __forceinline__ float sigmoid(float z) {
  z = z < -87.f ? -87.f : z;
  const float d = 1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f);
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

// ------------------------------------------------------------------ rows in registers
template <int LPR_, int NC_> struct Lanes {
  // a workgroup of four waves with several rows at a time, or one row's own
  static constexpr int LPR = LPR_, NC = NC_, NT = LPR > 64 ? LPR : 256, ROWS = NT / LPR;
};

// Sums of K values over a row's lanes, the same in all of them. red: K values
// for each wave, twice (a row uses one half, the next row the other).
template <class C, int K> __device__ __forceinline__ void row_sum(float (&x)[K], float (*red)[K], int tid) {
  constexpr int N = C::LPR < 64 ? C::LPR : 64, W = C::LPR / 64;
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lane_sum<N>(x[k]);
  if constexpr (W > 1) {
    if ((tid & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[tid >> 6][k] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) x[k] += red[w][k];
    }
  }
}

template <class C> constexpr int kWavesOf = C::NT / 64;

// A row's centred values and 1 / sqrt of their mean square.
template <bool BF16, class C, int V>
__device__ __forceinline__ void centre(float (&c)[C::NC][V], float &r, const Raw<BF16, V> (&x)[C::NC],
                                       const float (&one)[C::NC], const NormArgs &p, float inv,
                                       float (*red)[kWavesOf<C>][1], int tid) {
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) c[j][v] = x[j][v];
  }
  if (p.layer) {
#pragma unroll
    for (int j = 0; j < C::NC; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) s[0] += c[j][v];
    }
    row_sum<C>(s, red[0], tid);
    const float mean = s[0] * inv;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < C::NC; ++j) {  // one[j] is 0 past the row's end
#pragma unroll
      for (int v = 0; v < V; ++v) c[j][v] = __builtin_fmaf(-mean, one[j], c[j][v]);
    }
  }
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) s[0] = __builtin_fmaf(c[j][v], c[j][v], s[0]);
  }
  row_sum<C>(s, red[1], tid);
  r = 1.f / __builtin_sqrtf(s[0] * inv + p.eps);
}

template <bool BF16, int V, class C>
__device__ __forceinline__ void load_row(Raw<BF16, V> (&x)[C::NC], const void *p, int64_t row, const NormArgs &a,
                                         int l) {
  const char *base = static_cast<const char *>(p) + (size_t)row * a.D * sizeof(typename Elem<BF16>::T);
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
    const int col = (j * C::LPR + l) * V;
    x[j] = {};
    if (col < a.D) x[j] = load_raw<BF16, V>(base, col * (uint32_t)sizeof(typename Elem<BF16>::T));
  }
}

template <bool BF16, int V, class C>
__device__ __forceinline__ void store_row(void *p, int64_t row, const NormArgs &a, int l, const float (&y)[C::NC][V]) {
  char *base = static_cast<char *>(p) + (size_t)row * a.D * sizeof(typename Elem<BF16>::T);
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
    const int col = (j * C::LPR + l) * V;
    if (col < a.D) store_at<BF16>(base + col * (uint32_t)sizeof(typename Elem<BF16>::T), y[j]);
  }
}

template <int V, class C>
__device__ __forceinline__ void load_weights(float (&w)[C::NC][V], const void *p, const NormArgs &a, int l, float none) {
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (j * C::LPR + l) * V + v;
      w[j][v] = col < a.D ? load_w(p, col, a.wbf16, none) : 0.f;
    }
  }
}

template <bool BF16, bool GATE, int V, class C> __global__ __launch_bounds__(C::NT) void norm_forward_rows(NormArgs p) {
  constexpr int NC = C::NC;
  __shared__ float red[2][2][kWavesOf<C>][1];
  const int tid = threadIdx.x, l = tid % C::LPR;
  const float inv = 1.f / (float)p.D;
  float w[NC][V], b[NC][V], one[NC];
  load_weights<V, C>(w, p.weight, p, l, 1.f);
  load_weights<V, C>(b, p.bias, p, l, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) one[j] = (j * C::LPR + l) * V < p.D ? 1.f : 0.f;
  const int64_t step = (int64_t)gridDim.x * C::ROWS;
  int64_t row = (int64_t)blockIdx.x * C::ROWS + tid / C::LPR;
  Raw<BF16, V> x[NC], z[GATE ? NC : 1], xn[NC], zn[GATE ? NC : 1];
  if (row < p.rows) {
    load_row<BF16, V, C>(xn, p.x, row, p, l);
    if constexpr (GATE) load_row<BF16, V, C>(zn, p.gate, row, p, l);
  }
  for (int par = 0; row < p.rows; row += step, par ^= 1) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      x[j] = xn[j];
      if constexpr (GATE) z[j] = zn[j];
    }
    if (row + step < p.rows) {
      load_row<BF16, V, C>(xn, p.x, row + step, p, l);
      if constexpr (GATE) load_row<BF16, V, C>(zn, p.gate, row + step, p, l);
    }
    float c[NC][V], r;
    centre<BF16, C, V>(c, r, x, one, p, inv, red[par], tid);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[j][v] = __builtin_fmaf(c[j][v] * r, w[j][v], b[j][v]);
        if constexpr (GATE) {
          const float zv = z[j][v];
          c[j][v] *= zv * sigmoid(zv);
        }
      }
    }
    store_row<BF16, V, C>(p.y, row, p, l, c);
  }
}

template <bool BF16, bool GATE, int V, class C> __global__ __launch_bounds__(C::NT) void norm_backward_rows(NormArgs p) {
  constexpr int NC = C::NC;
  __shared__ float red[2][2][kWavesOf<C>][1], red2[2][kWavesOf<C>][2];
  const int tid = threadIdx.x, l = tid % C::LPR;
  const float inv = 1.f / (float)p.D;
  float w[NC][V], b[GATE ? NC : 1][V], one[NC], dw[NC][V] = {}, db[NC][V] = {};
  load_weights<V, C>(w, p.weight, p, l, 1.f);
  if constexpr (GATE) load_weights<V, C>(b, p.bias, p, l, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) one[j] = (j * C::LPR + l) * V < p.D ? 1.f : 0.f;
  const int64_t step = (int64_t)gridDim.x * C::ROWS;
  int64_t row = (int64_t)blockIdx.x * C::ROWS + tid / C::LPR;
  Raw<BF16, V> x[NC], y[NC], z[GATE ? NC : 1], xn[NC], yn[NC], zn[GATE ? NC : 1];
  if (row < p.rows) {
    load_row<BF16, V, C>(xn, p.x, row, p, l);
    load_row<BF16, V, C>(yn, p.dy, row, p, l);
    if constexpr (GATE) load_row<BF16, V, C>(zn, p.gate, row, p, l);
  }
  for (int par = 0; row < p.rows; row += step, par ^= 1) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      x[j] = xn[j];
      y[j] = yn[j];
      if constexpr (GATE) z[j] = zn[j];
    }
    if (row + step < p.rows) {
      load_row<BF16, V, C>(xn, p.x, row + step, p, l);
      load_row<BF16, V, C>(yn, p.dy, row + step, p, l);
      if constexpr (GATE) load_row<BF16, V, C>(zn, p.gate, row + step, p, l);
    }
    float c[NC][V], d[NC][V], r, s[2] = {0.f, 0.f};
    centre<BF16, C, V>(c, r, x, one, p, inv, red[par], tid);
    if constexpr (GATE) {
      float dz[NC][V];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float zv = z[j][v], sg = sigmoid(zv), yv = y[j][v];
          const float n = __builtin_fmaf(c[j][v] * r, w[j][v], b[j][v]);
          dz[j][v] = yv * n * (sg * __builtin_fmaf(zv, 1.f - sg, 1.f));
          d[j][v] = yv * (zv * sg);
        }
      }
      if (p.dgate) store_row<BF16, V, C>(p.dgate, row, p, l, dz);
    } else {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) d[j][v] = y[j][v];
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[j][v] *= r;  // xh
        dw[j][v] = __builtin_fmaf(d[j][v], c[j][v], dw[j][v]);
        db[j][v] += d[j][v];
        d[j][v] *= w[j][v];
        s[0] += d[j][v];
        s[1] = __builtin_fmaf(d[j][v], c[j][v], s[1]);
      }
    }
    row_sum<C>(s, red2[par], tid);
    const float md = p.layer ? s[0] * inv : 0.f, mx = s[1] * inv;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[j][v] = r * (__builtin_fmaf(-c[j][v], mx, d[j][v]) - md);
    }
    store_row<BF16, V, C>(p.dx, row, p, l, d);
  }
  // this workgroup's column sums: over its row groups, first inside a wave
  float *part = static_cast<float *>(p.workspace);
  if (!part) return;
  __shared__ float cols[4][C::LPR > 64 ? 1 : C::LPR * V];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? p.dbias : p.dweight)) continue;
    float *to = part + ((size_t)k * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float(&acc)[V] = k ? db[j] : dw[j];
      const int col = (j * C::LPR + l) * V;
      if constexpr (C::LPR > 64) {
        if (col < p.D) store_at<false>(reinterpret_cast<char *>(to + col), acc);
      } else {
#pragma unroll
        for (int off = C::LPR; off < 64; off <<= 1) {
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] += __shfl_xor(acc[v], off, 64);
        }
        __syncthreads();
        if ((tid & 63) < C::LPR) {
#pragma unroll
          for (int v = 0; v < V; ++v) cols[tid >> 6][l * V + v] = acc[v];
        }
        __syncthreads();
        for (int i = tid; i < C::LPR * V; i += C::NT) {
          const int at = j * C::LPR * V + i;
          if (at < p.D) to[at] = (cols[0][i] + cols[1][i]) + (cols[2][i] + cols[3][i]);
        }
      }
    }
  }
}

// ------------------------------------------------------------------ any width
constexpr int kNT = 256;

// Sum over the workgroup, the same value and rounding in every thread.
__device__ __forceinline__ float block_sum(float x, float *red, int tid) {
  x = lane_sum<64>(x);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// A row's statistics, the row read from memory for each pass.
template <bool BF16>
__device__ __forceinline__ void loop_stats(const typename Elem<BF16>::T *x, const NormArgs &p, float *red, int tid,
                                           float &mean, float &r) {
  float s = 0.f;
  mean = 0.f;
  if (p.layer) {
    for (int c = tid; c < p.D; c += kNT) s += Elem<BF16>::ld(x + c);
    mean = block_sum(s, red, tid) / (float)p.D;
    s = 0.f;
  }
  for (int c = tid; c < p.D; c += kNT) {
    const float v = Elem<BF16>::ld(x + c) - mean;
    s = __builtin_fmaf(v, v, s);
  }
  r = 1.f / __builtin_sqrtf(block_sum(s, red, tid) / (float)p.D + p.eps);
}

// Rows too wide for a workgroup's registers: one value a thread at a time.
template <bool BF16, bool GATE> __global__ __launch_bounds__(kNT) void norm_forward_loop(NormArgs p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  __shared__ float red[4];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + row * p.D;
    float mean, r;
    loop_stats<BF16>(x, p, red, tid, mean, r);
    for (int c = tid; c < p.D; c += kNT) {
      float y = (E::ld(x + c) - mean) * r * load_w(p.weight, c, p.wbf16, 1.f) + load_w(p.bias, c, p.wbf16, 0.f);
      if constexpr (GATE) {
        const float z = E::ld(static_cast<const T *>(p.gate) + row * p.D + c);
        y *= z * sigmoid(z);
      }
      E::st(static_cast<T *>(p.y) + row * p.D + c, y);
    }
  }
}

template <bool BF16, bool GATE> __global__ __launch_bounds__(kNT) void norm_backward_loop(NormArgs p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  __shared__ float red[4];
  const int tid = threadIdx.x;
  float *pw = static_cast<float *>(p.workspace) + (size_t)blockIdx.x * p.D;
  float *pb = static_cast<float *>(p.workspace) + ((size_t)gridDim.x + blockIdx.x) * p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + row * p.D, *dy = static_cast<const T *>(p.dy) + row * p.D;
    const T *gate = static_cast<const T *>(p.gate) + row * p.D;
    float mean, r, sd = 0.f, sx = 0.f;
    loop_stats<BF16>(x, p, red, tid, mean, r);
    for (int c = tid; c < p.D; c += kNT) {
      const float xh = (E::ld(x + c) - mean) * r, w = load_w(p.weight, c, p.wbf16, 1.f);
      float dn = E::ld(dy + c);
      if constexpr (GATE) {
        const float z = E::ld(gate + c), s = sigmoid(z), n = xh * w + load_w(p.bias, c, p.wbf16, 0.f);
        if (p.dgate) E::st(static_cast<T *>(p.dgate) + row * p.D + c, dn * n * (s * (1.f + z * (1.f - s))));
        dn *= z * s;
      }
      if (p.dweight) pw[c] = row == blockIdx.x ? dn * xh : pw[c] + dn * xh;
      if (p.dbias) pb[c] = row == blockIdx.x ? dn : pb[c] + dn;
      sd += dn * w;
      sx += dn * w * xh;
    }
    sd = p.layer ? block_sum(sd, red, tid) / (float)p.D : 0.f;
    sx = block_sum(sx, red, tid) / (float)p.D;
    for (int c = tid; c < p.D; c += kNT) {
      const float xh = (E::ld(x + c) - mean) * r;
      float dn = E::ld(dy + c);
      if constexpr (GATE) {
        const float z = E::ld(gate + c);
        dn *= z * sigmoid(z);
      }
      E::st(static_cast<T *>(p.dx) + row * p.D + c, r * (dn * load_w(p.weight, c, p.wbf16, 1.f) - xh * sx - sd));
    }
  }
}

// Column sums of the workgroups' partial sums, in a fixed order: 16 columns a
// workgroup, the parts over 64 groups of threads.
constexpr int kReduceNT = 1024;
__global__ __launch_bounds__(kReduceNT) void norm_reduce(NormArgs p, int parts) {
  __shared__ float red[64][17];
  const int tid = threadIdx.x, col = blockIdx.x * 16 + (tid & 15), grp = tid >> 4;
  void *out = blockIdx.y ? p.dbias : p.dweight;
  if (!out) return;
  const float *part = static_cast<const float *>(p.workspace) + (size_t)blockIdx.y * parts * p.D;
  float s = 0.f;
  if (col < p.D) {
#pragma unroll 8
    for (int g = grp; g < parts; g += 64) s += part[(size_t)g * p.D + col];
  }
  red[grp][tid & 15] = s;
  __syncthreads();
  for (int half = 32; half > 0; half >>= 1) {
    if (grp < half) red[grp][tid & 15] += red[grp + half][tid & 15];
    __syncthreads();
  }
  if (tid < 16 && col < p.D) store_w(out, col, p.wbf16, red[0][tid]);
}

// ------------------------------------------------------------------ which kernel
// The widest vectors every row of every tensor is aligned to (V values of at
// most 16 bytes), and the fewest lanes that hold a row with them; wider rows
// take more pieces a lane, then a whole workgroup. kLoop: too wide for that.
enum Plan { k2, k4, k8, k16, k32, k64, k128, k256, k512, k1024, k1024x2, k1024x4, kLoop };

struct How {
  Plan plan;
  int vec, rows, wgs;  // values a load, rows a workgroup holds at a time, workgroups at most
};

uintptr_t addresses(const NormArgs &p) {
  uintptr_t at = 0;
  for (const void *q : {p.x, p.gate, p.dy, (const void *)p.y, (const void *)p.dx, (const void *)p.dgate})
    at |= reinterpret_cast<uintptr_t>(q);
  return at;
}

How how(int D, bool bf16, uintptr_t at) {
  static constexpr struct { int most; Plan plan; int rows, wgs; bool narrow; } of[] = {
      {2, k2, 128, 1024, false},   {4, k4, 64, 1024, false},     {8, k8, 32, 1024, false},     {16, k16, 16, 1024, true},
      {32, k32, 8, 1024, false},   {64, k64, 4, 1024, true},     {128, k128, 1, 1024, false},  {256, k256, 1, 1024, true},
      {512, k512, 1, 512, false},  {1024, k1024, 1, 512, true},  {2048, k1024x2, 1, 512, false},
      {4096, k1024x4, 1, 256, true}};
  const int wide = bf16 ? 8 : 4;
  const bool aligned = D % wide == 0 && at % 16 == 0;
  const int vec = aligned ? wide : bf16 && D % 4 == 0 && at % 8 == 0 ? 4 : 1;
  const int n = (D + vec - 1) / vec;
  for (const auto &o : of)
    if (n <= o.most && (aligned ? o.plan != k1024x4 : o.narrow)) return How{o.plan, vec, o.rows, o.wgs};
  return How{kLoop, 1, 1, 1024};
}

int64_t groups(const How &h, int64_t rows) {
  const int64_t need = (rows + h.rows - 1) / h.rows;
  return need < h.wgs ? need : h.wgs;
}

template <bool BF16, bool GATE, bool BACK, int V, class C> void go(const NormArgs &p, unsigned grid, hipStream_t st) {
  if constexpr (BACK)
    hipLaunchKernelGGL((norm_backward_rows<BF16, GATE, V, C>), dim3(grid), dim3(C::NT), 0, st, p);
  else
    hipLaunchKernelGGL((norm_forward_rows<BF16, GATE, V, C>), dim3(grid), dim3(C::NT), 0, st, p);
}

// V narrower than 16 bytes: fewer lane counts, each for a wider range.
template <bool BF16, bool GATE, bool BACK, int V> bool go_narrow(const NormArgs &p, Plan plan, unsigned grid, hipStream_t st) {
  switch (plan) {
    case k16: return go<BF16, GATE, BACK, V, Lanes<16, 1>>(p, grid, st), true;
    case k64: return go<BF16, GATE, BACK, V, Lanes<64, 1>>(p, grid, st), true;
    case k256: return go<BF16, GATE, BACK, V, Lanes<256, 1>>(p, grid, st), true;
    case k1024: return go<BF16, GATE, BACK, V, Lanes<1024, 1>>(p, grid, st), true;
    case k1024x4: return go<BF16, GATE, BACK, V, Lanes<1024, 4>>(p, grid, st), true;
    default: return false;
  }
}

template <bool BF16, bool GATE, bool BACK> void launch_g(const NormArgs &p, const How &h, unsigned grid, hipStream_t st) {
  constexpr int W = BF16 ? 8 : 4;
  if (h.vec == W) {
    switch (h.plan) {
      case k2: return go<BF16, GATE, BACK, W, Lanes<2, 1>>(p, grid, st);
      case k4: return go<BF16, GATE, BACK, W, Lanes<4, 1>>(p, grid, st);
      case k8: return go<BF16, GATE, BACK, W, Lanes<8, 1>>(p, grid, st);
      case k16: return go<BF16, GATE, BACK, W, Lanes<16, 1>>(p, grid, st);
      case k32: return go<BF16, GATE, BACK, W, Lanes<32, 1>>(p, grid, st);
      case k64: return go<BF16, GATE, BACK, W, Lanes<64, 1>>(p, grid, st);
      case k128: return go<BF16, GATE, BACK, W, Lanes<128, 1>>(p, grid, st);
      case k256: return go<BF16, GATE, BACK, W, Lanes<256, 1>>(p, grid, st);
      case k512: return go<BF16, GATE, BACK, W, Lanes<512, 1>>(p, grid, st);
      case k1024: return go<BF16, GATE, BACK, W, Lanes<1024, 1>>(p, grid, st);
      default: return go<BF16, GATE, BACK, W, Lanes<1024, 2>>(p, grid, st);
    }
  }
  if constexpr (BF16) {
    if (h.vec == 4 && go_narrow<BF16, GATE, BACK, 4>(p, h.plan, grid, st)) return;
  }
  if (h.vec == 1 && go_narrow<BF16, GATE, BACK, 1>(p, h.plan, grid, st)) return;
  if constexpr (BACK)
    hipLaunchKernelGGL((norm_backward_loop<BF16, GATE>), dim3(grid), dim3(kNT), 0, st, p);
  else
    hipLaunchKernelGGL((norm_forward_loop<BF16, GATE>), dim3(grid), dim3(kNT), 0, st, p);
}

}  // namespace

#ifdef GDN2_NORM_BACKWARD
size_t norm_backward_workspace_bytes(int64_t rows, int D) {
  // the most workgroups of any way to take the rows
  return (size_t)(rows < 1024 ? rows : 1024) * D * 2 * sizeof(float);
}

hipError_t launch_norm_backward(const NormArgs &q, hipStream_t st) {
  NormArgs p = q;
  if (!p.dweight && !p.dbias) p.workspace = nullptr;
  const How h = how(p.D, p.bf16, addresses(p));
  const int64_t parts = groups(h, p.rows);
  if (parts > 0) {
    const unsigned g = (unsigned)parts;
    if (p.bf16)
      p.gate ? launch_g<true, true, true>(p, h, g, st) : launch_g<true, false, true>(p, h, g, st);
    else
      p.gate ? launch_g<false, true, true>(p, h, g, st) : launch_g<false, false, true>(p, h, g, st);
  }
  if (p.dweight || p.dbias)
    hipLaunchKernelGGL(norm_reduce, dim3((unsigned)((p.D + 15) / 16), 2), dim3(kReduceNT), 0, st, p, (int)parts);
  return hipGetLastError();
}
#else
hipError_t launch_norm_forward(const NormArgs &p, hipStream_t st) {
  const How h = how(p.D, p.bf16, addresses(p));
  const unsigned g = (unsigned)groups(h, p.rows);
  if (p.bf16)
    p.gate ? launch_g<true, true, false>(p, h, g, st) : launch_g<true, false, false>(p, h, g, st);
  else
    p.gate ? launch_g<false, true, false>(p, h, g, st) : launch_g<false, false, false>(p, h, g, st);
  return hipGetLastError();
}
#endif

}  // namespace gdn2
