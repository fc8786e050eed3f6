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
// that a large common offset costs the mean's own rounding and no more. All sums
// are fp32.
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

// s = 1 / (1 + e^-z) of a gate z. Below -87 (s is 2e-38 there) a gate is closed:
// s is 0 and z comes back as -87, so that z s and its derivative are 0 however
// low z is, -inf too. NaN stays.
__device__ __forceinline__ float sigmoid(float &z) {
  const bool closed = z < -87.f;
  z = closed ? -87.f : z;
  const float d = 1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f);
  const float r = __builtin_amdgcn_rcpf(d);
  return closed ? 0.f : __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}
// The derivative of z s from it and s; s is 1 long before z s is 88, so 88 stands
// for all above it (inf * 0).
__device__ __forceinline__ float silu_slope(float zs, float s) {
  return __builtin_fmaf(__builtin_fminf(zs, 88.f), 1.f - s, s);
}

// ------------------------------------------------------------------ rows in registers
// A row on LPR lanes of a wave, a workgroup of four waves taking several rows
// at a time; or (LPR = kBlock) on the whole of a workgroup of any number of
// waves, one row at a time.
constexpr int kBlock = 1024;
template <int LPR_, int NC_> struct Lanes {
  static constexpr int LPR = LPR_, NC = NC_, NT = LPR == kBlock ? kBlock : 256, ROWS = NT / LPR, WAVES = NT / 64;
  static constexpr bool BLOCK = LPR == kBlock;
  static __device__ __forceinline__ int lanes() { return BLOCK ? (int)blockDim.x : LPR; }
  static __device__ __forceinline__ int lane(int tid) { return BLOCK ? tid : tid % LPR; }
  static __device__ __forceinline__ int group(int tid) { return BLOCK ? 0 : tid / LPR; }
};

// Sums of K values over a row's lanes, the same in all of them. red: K values
// for each wave, twice (a row uses one half, the next row the other).
template <class C, int K> __device__ __forceinline__ void row_sum(float (&x)[K], float (*red)[K], int tid) {
  constexpr int N = C::BLOCK ? 64 : C::LPR;
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lane_sum<N>(x[k]);
  if constexpr (C::BLOCK) {  // at most 16 waves' sums, one a lane of every 16
    if ((tid & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[tid >> 6][k] = x[k];
    }
    __syncthreads();
    const int w = tid & 15;
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = lane_sum<16>(w < (int)(blockDim.x >> 6) ? red[w][k] : 0.f);
  }
}

// A row's centred values and 1 / sqrt of their mean square.
template <bool BF16, class C, int V>
__device__ __forceinline__ void centre(float (&c)[C::NC][V], float &r, const Raw<BF16, V> (&x)[C::NC],
                                       const float (&one)[C::NC], const NormArgs &p, float inv,
                                       float (*red)[C::WAVES][1], int tid) {
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
    const int col = (j * C::lanes() + l) * V;
    x[j] = {};
    if (col < a.D) x[j] = load_raw<BF16, V>(base, col * (uint32_t)sizeof(typename Elem<BF16>::T));
  }
}

// Piece j of a lane's row.
template <bool BF16, int V, class C>
__device__ __forceinline__ void store_piece(void *p, int64_t row, int j, const NormArgs &a, int l, const float (&y)[V]) {
  char *base = static_cast<char *>(p) + (size_t)row * a.D * sizeof(typename Elem<BF16>::T);
  const int col = (j * C::lanes() + l) * V;
  if (col < a.D) store_at<BF16>(base + col * (uint32_t)sizeof(typename Elem<BF16>::T), y);
}

template <bool BF16, int V, class C>
__device__ __forceinline__ void store_row(void *p, int64_t row, const NormArgs &a, int l, const float (&y)[C::NC][V]) {
#pragma unroll
  for (int j = 0; j < C::NC; ++j) store_piece<BF16, V, C>(p, row, j, a, l, y[j]);
}

template <int V, class C>
__device__ __forceinline__ void load_weights(float (&w)[C::NC][V], const void *p, const NormArgs &a, int l, float none) {
#pragma unroll
  for (int j = 0; j < C::NC; ++j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int col = (j * C::lanes() + l) * V + v;
      w[j][v] = col < a.D ? load_w(p, col, a.wbf16, none) : 0.f;
    }
  }
}

template <bool BF16, bool GATE, int V, class C> __global__ __launch_bounds__(C::NT) void norm_forward_rows(NormArgs p) {
  constexpr int NC = C::NC;
  __shared__ float red[2][2][C::WAVES][1];
  const int tid = threadIdx.x, l = C::lane(tid);
  const float inv = 1.f / (float)p.D;
  float w[NC][V], b[NC][V], one[NC];
  load_weights<V, C>(w, p.weight, p, l, 1.f);
  load_weights<V, C>(b, p.bias, p, l, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) one[j] = (j * C::lanes() + l) * V < p.D ? 1.f : 0.f;
  const int64_t step = (int64_t)gridDim.x * C::ROWS;
  int64_t row = (int64_t)blockIdx.x * C::ROWS + C::group(tid);
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
          float zv = z[j][v];
          const float sg = sigmoid(zv);
          c[j][v] *= zv * sg;
        }
      }
    }
    store_row<BF16, V, C>(p.y, row, p, l, c);
  }
}

template <bool BF16, bool GATE, int V, class C> __global__ __launch_bounds__(C::NT) void norm_backward_rows(NormArgs p) {
  constexpr int NC = C::NC;
  // the next row's loads in flight; not with 16 values a lane, where 1024
  // threads have no registers for them (270 us instead of 127 at 4096 x 16384;
  // with a gate even without them 156 bytes a lane go to memory, 240 us)
  constexpr bool AHEAD = NC * V <= 8;
  __shared__ float red[2][2][C::WAVES][1], red2[2][C::WAVES][2];
  const int tid = threadIdx.x, l = C::lane(tid);
  const float inv = 1.f / (float)p.D;
  float w[NC][V], b[GATE ? NC : 1][V], one[NC], dw[NC][V] = {}, db[NC][V] = {};
  load_weights<V, C>(w, p.weight, p, l, 1.f);
  if constexpr (GATE) load_weights<V, C>(b, p.bias, p, l, 0.f);
#pragma unroll
  for (int j = 0; j < NC; ++j) one[j] = (j * C::lanes() + l) * V < p.D ? 1.f : 0.f;
  const int64_t step = (int64_t)gridDim.x * C::ROWS;
  int64_t row = (int64_t)blockIdx.x * C::ROWS + C::group(tid);
  Raw<BF16, V> x[NC], y[NC], z[GATE ? NC : 1], xn[NC], yn[NC], zn[GATE ? NC : 1];
  auto load = [&](int64_t at) {
    load_row<BF16, V, C>(xn, p.x, at, p, l);
    load_row<BF16, V, C>(yn, p.dy, at, p, l);
    if constexpr (GATE) load_row<BF16, V, C>(zn, p.gate, at, p, l);
  };
  if (AHEAD && row < p.rows) load(row);
  for (int par = 0; row < p.rows; row += step, par ^= 1) {
    if (!AHEAD) load(row);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      x[j] = xn[j];
      y[j] = yn[j];
      if constexpr (GATE) z[j] = zn[j];
    }
    if (AHEAD && row + step < p.rows) load(row + step);
    float c[NC][V], d[NC][V], r, s[2] = {0.f, 0.f};
    centre<BF16, C, V>(c, r, x, one, p, inv, red[par], tid);
    if constexpr (GATE) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float dz[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float zv = z[j][v];
          const float sg = sigmoid(zv), zs = zv * sg, yv = y[j][v];
          const float n = __builtin_fmaf(c[j][v] * r, w[j][v], b[j][v]);
          dz[v] = yv * n * silu_slope(zs, sg);
          d[j][v] = yv * zs;
        }
        if (p.dgate) store_piece<BF16, V, C>(p.dgate, row, j, p, l, dz);
      }
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
  __shared__ float cols[4][C::BLOCK ? 1 : C::LPR * V];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? p.dbias : p.dweight)) continue;
    float *to = part + ((size_t)k * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float(&acc)[V] = k ? db[j] : dw[j];
      const int col = (j * C::lanes() + l) * V;
      if constexpr (C::BLOCK) {
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
// Rows too wide for registers: a workgroup a row, read from memory (or the
// caches) again for each of its sums, V values (4 or 1) a thread at a time.
template <bool BF16, int V>
__device__ __forceinline__ void loop_stats(const typename Elem<BF16>::T *x, const NormArgs &p,
                                           float (*red)[kBlock / 64][1], int tid, float &mean, float &r) {
  using C = Lanes<kBlock, 1>;
  float s[1] = {0.f}, f[V];
  mean = 0.f;
  if (p.layer) {
    for (int c = tid * V; c < p.D; c += kBlock * V) {
      load_f<BF16>(f, x, c);
#pragma unroll
      for (int v = 0; v < V; ++v) s[0] += f[v];
    }
    row_sum<C>(s, red[0], tid);
    mean = s[0] / (float)p.D;
    s[0] = 0.f;
  }
  for (int c = tid * V; c < p.D; c += kBlock * V) {
    load_f<BF16>(f, x, c);
#pragma unroll
    for (int v = 0; v < V; ++v) s[0] = __builtin_fmaf(f[v] - mean, f[v] - mean, s[0]);
  }
  row_sum<C>(s, red[1], tid);
  r = 1.f / __builtin_sqrtf(s[0] / (float)p.D + p.eps);
}

template <bool BF16, bool GATE, int V> __global__ __launch_bounds__(kBlock) void norm_forward_loop(NormArgs p) {
  using T = typename Elem<BF16>::T;
  __shared__ float red[2][2][kBlock / 64][1];
  const int tid = threadIdx.x;
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
    const T *x = static_cast<const T *>(p.x) + row * p.D;
    float mean, r, f[V], z[V];
    loop_stats<BF16, V>(x, p, red[par], tid, mean, r);
    for (int c = tid * V; c < p.D; c += kBlock * V) {
      load_f<BF16>(f, x, c);
      if constexpr (GATE) load_f<BF16>(z, p.gate, (size_t)row * p.D + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f[v] = (f[v] - mean) * r * load_w(p.weight, c + v, p.wbf16, 1.f) + load_w(p.bias, c + v, p.wbf16, 0.f);
        if constexpr (GATE) {
          const float sg = sigmoid(z[v]);
          f[v] *= z[v] * sg;
        }
      }
      store_f<BF16>(p.y, (size_t)row * p.D + c, f);
    }
  }
}

template <bool BF16, bool GATE, int V> __global__ __launch_bounds__(kBlock) void norm_backward_loop(NormArgs p) {
  using T = typename Elem<BF16>::T;
  using C = Lanes<kBlock, 1>;
  __shared__ float red[2][2][kBlock / 64][1], red2[2][kBlock / 64][2];
  const int tid = threadIdx.x;
  // this workgroup's column sums, added to row by row: each by one thread
  float *pw = static_cast<float *>(p.workspace) + (size_t)blockIdx.x * p.D;
  float *pb = static_cast<float *>(p.workspace) + ((size_t)gridDim.x + blockIdx.x) * p.D;
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
    const size_t at = (size_t)row * p.D;
    const T *x = static_cast<const T *>(p.x) + at;
    const bool first = row == blockIdx.x;
    float mean, r, s[2] = {0.f, 0.f}, f[V], d[V], z[V], acc[V];
    loop_stats<BF16, V>(x, p, red[par], tid, mean, r);
    for (int c = tid * V; c < p.D; c += kBlock * V) {
      load_f<BF16>(f, x, c);
      load_f<BF16>(d, p.dy, at + c);
      if constexpr (GATE) load_f<BF16>(z, p.gate, at + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        f[v] = (f[v] - mean) * r;
        const float w = load_w(p.weight, c + v, p.wbf16, 1.f);
        if constexpr (GATE) {
          const float sg = sigmoid(z[v]), n = f[v] * w + load_w(p.bias, c + v, p.wbf16, 0.f), dz = d[v] * n;
          const float zs = z[v] * sg;
          d[v] *= zs;
          z[v] = dz * silu_slope(zs, sg);
        }
        s[0] += d[v] * w;
        s[1] += d[v] * w * f[v];
      }
      if constexpr (GATE) {
        if (p.dgate) store_f<BF16>(p.dgate, at + c, z);
      }
      if (p.dweight) {
        if (!first) load_f<false>(acc, pw, c);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = first ? d[v] * f[v] : acc[v] + d[v] * f[v];
        store_f<false>(pw, c, acc);
      }
      if (p.dbias) {
        if (!first) load_f<false>(acc, pb, c);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = first ? d[v] : acc[v] + d[v];
        store_f<false>(pb, c, acc);
      }
    }
    row_sum<C>(s, red2[par], tid);
    const float md = p.layer ? s[0] / (float)p.D : 0.f, mx = s[1] / (float)p.D;
    for (int c = tid * V; c < p.D; c += kBlock * V) {
      load_f<BF16>(f, x, c);
      load_f<BF16>(d, p.dy, at + c);
      if constexpr (GATE) load_f<BF16>(z, p.gate, at + c);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (GATE) {
          const float sg = sigmoid(z[v]);
          d[v] *= z[v] * sg;
        }
        d[v] = r * (d[v] * load_w(p.weight, c + v, p.wbf16, 1.f) - (f[v] - mean) * r * mx - md);
      }
      store_f<BF16>(p.dx, at + c, d);
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
// V: the widest vectors that every row of every tensor is aligned to (at most
// 16 bytes). A row of up to 64 of them lies on the fewest lanes of a wave that
// hold it, a wider one on a workgroup of as many waves as it needs, with two a
// lane where it has more than 256 (8192 x 8192 bf16, forward: 55 us, with one
// 68; at 256 the two are even) or they are of 8 bytes; single values go four to
// a lane. kLoop: rows too
// wide for that.
enum Plan { k2, k4, k8, k16, k32, k64, k16x4, k64x4, kRow, kRow2, kRow4, kLoop };

struct How {
  Plan plan;
  int vec, rows, threads;  // values a load; of a workgroup: rows at a time, threads
};

uintptr_t addresses(const NormArgs &p) {
  uintptr_t at = 0;
  for (const void *q : {p.x, p.gate, p.dy, (const void *)p.y, (const void *)p.dx, (const void *)p.dgate})
    at |= reinterpret_cast<uintptr_t>(q);
  return at;
}

// pairs: whether a lane's registers hold two vectors well (not with a gate in
// the backward, 137 against 304 us at 16384 x 4096).
How how(int D, bool bf16, uintptr_t at, bool pairs) {
  const int wide = bf16 ? 8 : 4;
  const bool aligned = D % wide == 0 && at % 16 == 0;
  const int vec = aligned ? wide : bf16 && D % 4 == 0 && at % 8 == 0 ? 4 : 1;
  const int n = (D + vec - 1) / vec;
  auto row = [&](Plan plan, int nc) { return How{plan, vec, 1, ((n + nc - 1) / nc + 63) / 64 * 64}; };
  if (vec == 1) {
    if (n <= 16) return How{k16, vec, 16, 256};
    if (n <= 64) return How{k16x4, vec, 16, 256};
    if (n <= 256) return How{k64x4, vec, 4, 256};
    if (n <= 4 * kBlock) return row(kRow4, 4);
  } else {
    int lanes = aligned ? 2 : 16, plan = aligned ? k2 : k16;
    for (; lanes < n && lanes < 64; lanes *= 2) ++plan;
    if (n <= 64) return How{(Plan)plan, vec, 256 / lanes, 256};
    if (aligned && n <= (pairs ? 256 : kBlock)) return row(kRow, 1);
    if (n <= 2 * kBlock) return row(kRow2, 2);
  }
  return How{kLoop, vec, 1, kBlock};
}

// Workgroups: 1024 threads for each compute unit (a half and the double of it
// measured slower on most of twelve shapes, forward and backward).
int64_t groups(const How &h, int64_t rows) {
  const int64_t need = (rows + h.rows - 1) / h.rows, most = 256 * 1024 / h.threads;
  return need < most ? need : most;
}

template <bool BF16, bool GATE, bool BACK, int V, class C>
void go(const NormArgs &p, const How &h, unsigned grid, hipStream_t st) {
  if constexpr (BACK)
    hipLaunchKernelGGL((norm_backward_rows<BF16, GATE, V, C>), dim3(grid), dim3(h.threads), 0, st, p);
  else
    hipLaunchKernelGGL((norm_forward_rows<BF16, GATE, V, C>), dim3(grid), dim3(h.threads), 0, st, p);
}

template <bool BF16, bool GATE, bool BACK, int V> void go_loop(const NormArgs &p, unsigned grid, hipStream_t st) {
  if constexpr (BACK)
    hipLaunchKernelGGL((norm_backward_loop<BF16, GATE, V>), dim3(grid), dim3(kBlock), 0, st, p);
  else
    hipLaunchKernelGGL((norm_forward_loop<BF16, GATE, V>), dim3(grid), dim3(kBlock), 0, st, p);
}

template <bool BF16, bool GATE, bool BACK> void launch_g(const NormArgs &p, const How &h, unsigned grid, hipStream_t st) {
  constexpr int W = BF16 ? 8 : 4;
  if (h.plan != kLoop && h.vec == W) {
    switch (h.plan) {
      case k2: return go<BF16, GATE, BACK, W, Lanes<2, 1>>(p, h, grid, st);
      case k4: return go<BF16, GATE, BACK, W, Lanes<4, 1>>(p, h, grid, st);
      case k8: return go<BF16, GATE, BACK, W, Lanes<8, 1>>(p, h, grid, st);
      case k16: return go<BF16, GATE, BACK, W, Lanes<16, 1>>(p, h, grid, st);
      case k32: return go<BF16, GATE, BACK, W, Lanes<32, 1>>(p, h, grid, st);
      case k64: return go<BF16, GATE, BACK, W, Lanes<64, 1>>(p, h, grid, st);
      case kRow: return go<BF16, GATE, BACK, W, Lanes<kBlock, 1>>(p, h, grid, st);
      default: return go<BF16, GATE, BACK, W, Lanes<kBlock, 2>>(p, h, grid, st);
    }
  }
  if constexpr (BF16) {
    if (h.plan != kLoop && h.vec == 4) {
      switch (h.plan) {
        case k16: return go<BF16, GATE, BACK, 4, Lanes<16, 1>>(p, h, grid, st);
        case k32: return go<BF16, GATE, BACK, 4, Lanes<32, 1>>(p, h, grid, st);
        case k64: return go<BF16, GATE, BACK, 4, Lanes<64, 1>>(p, h, grid, st);
        default: return go<BF16, GATE, BACK, 4, Lanes<kBlock, 2>>(p, h, grid, st);
      }
    }
  }
  if (h.plan != kLoop) {
    switch (h.plan) {
      case k16: return go<BF16, GATE, BACK, 1, Lanes<16, 1>>(p, h, grid, st);
      case k16x4: return go<BF16, GATE, BACK, 1, Lanes<16, 4>>(p, h, grid, st);
      case k64x4: return go<BF16, GATE, BACK, 1, Lanes<64, 4>>(p, h, grid, st);
      default: return go<BF16, GATE, BACK, 1, Lanes<kBlock, 4>>(p, h, grid, st);
    }
  }
  if (h.vec > 1) return go_loop<BF16, GATE, BACK, 4>(p, grid, st);
  go_loop<BF16, GATE, BACK, 1>(p, grid, st);
}

}  // namespace

#ifdef GDN2_NORM_BACKWARD
size_t norm_backward_workspace_bytes(int64_t rows, int D, bool bf16) {
  // whatever the tensors' alignment, with a gate or without
  int64_t most = 0;
  for (uintptr_t at : {0, 8, 2}) {
    for (bool pairs : {false, true}) {
      const int64_t g = groups(how(D, bf16, at, pairs), rows);
      most = g > most ? g : most;
    }
  }
  return (size_t)most * D * 2 * sizeof(float);
}

hipError_t launch_norm_backward(const NormArgs &q, hipStream_t st) {
  NormArgs p = q;
  if (!p.dweight && !p.dbias) p.workspace = nullptr;
  const How h = how(p.D, p.bf16, addresses(p), !p.gate);
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
  const How h = how(p.D, p.bf16, addresses(p), true);
  const unsigned g = (unsigned)groups(h, p.rows);
  if (p.bf16)
    p.gate ? launch_g<true, true, false>(p, h, g, st) : launch_g<true, false, false>(p, h, g, st);
  else
    p.gate ? launch_g<false, true, false>(p, h, g, st) : launch_g<false, false, false>(p, h, g, st);
  return hipGetLastError();
}
#endif

}  // namespace gdn2
