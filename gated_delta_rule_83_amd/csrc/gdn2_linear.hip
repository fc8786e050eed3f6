// gdn2_linear.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t x_t,
// channel by channel, its gradients, and its single-token step.
//
// A token is the map h -> a h + u (u = b x); maps compose:
//   (a2, u2) after (a1, u1) = (a2 a1, a2 u1 + u2).
// A workgroup of 256 threads owns 64 channels and holds 128 tokens of them in
// registers: VEC channels (one wide load) by L = 128 / slots consecutive
// tokens a thread. It composes each thread's tokens, scans the threads' maps
// (lane shuffles inside a wave, LDS across the four waves), and walks its
// tokens again from the state that enters them. Everything between the loads
// and the one rounding of an output is fp32.
#include "gdn2_device.hpp"
#include "gdn2_linear.hpp"

#include "gdn2.h"

#include <initializer_list>

namespace gdn2 {

namespace {

constexpr int kNT = 256;

template <class T, int N> struct alignas(sizeof(T) * N) Vec { T e[N]; };

template <bool BF16, int N>
__device__ __forceinline__ void load_f(float (&f)[N], const void *p, size_t i) {
  using T = typename Elem<BF16>::T;
  const Vec<T, N> v = *reinterpret_cast<const Vec<T, N> *>(static_cast<const T *>(p) + i);
#pragma unroll
  for (int c = 0; c < N; ++c) f[c] = Elem<BF16>::f(v.e[c]);
}

template <bool BF16, int N>
__device__ __forceinline__ void store_f(void *p, size_t i, const float (&f)[N]) {
  using T = typename Elem<BF16>::T;
  Vec<T, N> v;
#pragma unroll
  for (int c = 0; c < N; ++c) Elem<BF16>::st(&v.e[c], f[c]);
  *reinterpret_cast<Vec<T, N> *>(static_cast<T *>(p) + i) = v;
}

// 1 / d for d >= 1 (v_rcp_f32 and one Newton step: within 1 ulp).
__device__ __forceinline__ float recip(float d) {
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

// p = 1 / (1 + e^x) and q = 1 - p = e^x / (1 + e^x), neither by a difference:
// both keep their relative accuracy however near the other is to 1. |x| above
// 87 counts as 87, where e^x is still finite and p or q below 2e-38; NaN stays.
__device__ __forceinline__ void split_sigmoid(float x, float &p, float &q) {
  x = x > 87.f ? 87.f : x;
  x = x < -87.f ? -87.f : x;
  const float e = __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
  p = recip(1.f + e);
  q = e * p;
}

template <int FORM> struct Form {
  static constexpr bool pre = FORM == GDN2_LINEAR_PREACT || FORM == GDN2_LINEAR_TIED_PREACT;
  static constexpr bool tied = FORM == GDN2_LINEAR_TIED || FORM == GDN2_LINEAR_TIED_PREACT;
};

// The gates of one token from what was loaded for them: decay a, input gate b.
template <int FORM, int N>
__device__ __forceinline__ void activate(float (&a)[N], float (&b)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    if constexpr (Form<FORM>::pre) {
      float q;
      split_sigmoid(a[c], a[c], q);
      if constexpr (Form<FORM>::tied) {
        b[c] = q;
      } else {
        split_sigmoid(-b[c], b[c], q);
      }
    } else if constexpr (Form<FORM>::tied) {
      b[c] = 1.f - a[c];
    }
  }
}

struct Lin {
  const void *x, *a, *b;
  const float *h0;
  void *o;
  float *h_T, *ck;
  const void *dO;
  const float *dh_T;
  void *dx, *da, *db;
  float *dh0;
  const int32_t *cu;
  int B, T, D, nblk;
};

__device__ __forceinline__ int clamp_offset(int x, int T) { return x < 0 ? 0 : x > T ? T : x; }

// Geometry of a thread: ct-th group of VEC channels, s-th slot of L tokens.
template <int VEC> struct Geo {
  static constexpr int CT = kLinChannels / VEC, NS = kNT / CT, L = kLinTile / NS, WS = 64 / CT;  // WS: slots a wave
};

// Scan of the threads' maps (A, U) in token order (or, REV, from the last
// token to the first): on return (A, U) is the map of all earlier threads of
// this wave, and tot[w] in LDS the whole map of wave w.
template <int VEC, bool REV>
__device__ __forceinline__ void wave_scan(float (&A)[VEC], float (&U)[VEC], float2 (*tot)[kLinChannels], int tid) {
  using G = Geo<VEC>;
  const int lane = tid & 63, w = tid >> 6, ct = lane % G::CT, sl = lane / G::CT;
#pragma unroll
  for (int off = 1; off < G::WS; off <<= 1) {
    const bool has = REV ? sl + off < G::WS : sl >= off;
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      const float pa = REV ? __shfl_down(A[c], off * G::CT, 64) : __shfl_up(A[c], off * G::CT, 64);
      const float pu = REV ? __shfl_down(U[c], off * G::CT, 64) : __shfl_up(U[c], off * G::CT, 64);
      if (has) {
        U[c] = __builtin_fmaf(A[c], pu, U[c]);
        A[c] *= pa;
      }
    }
  }
  if (sl == (REV ? 0 : G::WS - 1)) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) tot[w][ct * VEC + c] = float2{A[c], U[c]};
  }
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    if constexpr (G::WS == 1) {
      A[c] = 1.f;
      U[c] = 0.f;
    } else {
      const float pa = REV ? __shfl_down(A[c], G::CT, 64) : __shfl_up(A[c], G::CT, 64);
      const float pu = REV ? __shfl_down(U[c], G::CT, 64) : __shfl_up(U[c], G::CT, 64);
      const bool first = REV ? sl == G::WS - 1 : sl == 0;
      A[c] = first ? 1.f : pa;
      U[c] = first ? 0.f : pu;
    }
  }
}

// The value entering this thread's tokens and the value leaving the tile,
// from the value entering the tile (carry, replaced by the leaving one).
template <int VEC, bool REV>
__device__ __forceinline__ void enter(float (&in)[VEC], float (&carry)[VEC], const float (&A)[VEC],
                                      const float (&U)[VEC], const float2 (*tot)[kLinChannels], int tid) {
  using G = Geo<VEC>;
  const int w = tid >> 6, ct = (tid & 63) % G::CT;
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    float h = carry[c], mine = h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = REV ? 3 - i : i;
      if (j == w) mine = h;
      const float2 t = tot[j][ct * VEC + c];
      h = __builtin_fmaf(t.x, h, t.y);
    }
    in[c] = __builtin_fmaf(A[c], mine, U[c]);
    carry[c] = h;
  }
}

// One workgroup per (sequence, 64 channels), tile after tile. Tiles lie on
// multiples of 128 of the token axis (packed sequences: of the packed axis),
// so that the saved states' rows are the same whatever the sequences.
template <bool BF16, int FORM, int VEC>
__global__ __launch_bounds__(kNT) void linear_forward_seq(Lin p) {
  using G = Geo<VEC>;
  constexpr bool GB = BF16 && Form<FORM>::pre;  // gates in bf16
  __shared__ float2 tot[2][4][kLinChannels];
  const int tid = threadIdx.x, ct = tid % G::CT, s = tid / G::CT;
  const int n = blockIdx.x / p.nblk, blk = blockIdx.x - n * p.nblk;
  const int D = p.D, c0 = blk * kLinChannels + ct * VEC;
  const bool own = c0 < D;
  const int cc = own ? c0 : D - VEC;  // a channel to read in any case
  int lo = 0, hi = p.T;
  size_t row0 = (size_t)n * p.T;
  if (p.cu) {
    lo = clamp_offset(p.cu[n], p.T);
    hi = clamp_offset(p.cu[n + 1], p.T);
    row0 = 0;
  }
  const size_t ck0 = p.cu ? 0 : (size_t)n * ((p.T + kLinTile - 1) / kLinTile);
  float carry[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) carry[c] = p.h0 ? p.h0[(size_t)n * D + cc + c] : 0.f;
  int par = 0;
  for (int t0 = hi > lo ? lo - lo % kLinTile : hi; t0 < hi; t0 += kLinTile, par ^= 1) {
    if (p.ck && own && s == 0 && t0 > lo) store_f<false>(p.ck, (ck0 + t0 / kLinTile) * D + c0, carry);
    float a[G::L][VEC], u[G::L][VEC];
    const int ts = t0 + s * G::L;
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int t = ts + i, tc = t < lo ? lo : t >= hi ? hi - 1 : t;
      const size_t at = (row0 + tc) * D + cc;
      float b[VEC];
      load_f<BF16>(u[i], p.x, at);
      load_f<GB>(a[i], p.a, at);
      if constexpr (!Form<FORM>::tied) load_f<GB>(b, p.b, at);
      activate<FORM>(a[i], b);
      const bool in = t == tc;  // outside the sequence: the identity map
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        u[i][c] = in ? b[c] * u[i][c] : 0.f;
        a[i][c] = in ? a[i][c] : 1.f;
      }
    }
    float A[VEC], U[VEC], h[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      A[c] = a[0][c];
      U[c] = u[0][c];
    }
#pragma unroll
    for (int i = 1; i < G::L; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        U[c] = __builtin_fmaf(a[i][c], U[c], u[i][c]);
        A[c] *= a[i][c];
      }
    }
    wave_scan<VEC, false>(A, U, tot[par], tid);
    __syncthreads();
    enter<VEC, false>(h, carry, A, U, tot[par], tid);
    if (p.o) {
#pragma unroll
      for (int i = 0; i < G::L; ++i) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) h[c] = __builtin_fmaf(a[i][c], h[c], u[i][c]);
        const int t = ts + i;
        if (own && t >= lo && t < hi) store_f<BF16>(p.o, (row0 + t) * D + c0, h);
      }
    }
  }
  if (p.h_T && own && s == 0) store_f<false>(p.h_T, (size_t)n * D + c0, carry);
}

// Gradients. With m the adjoint of the state between two tokens (dh_T after
// the last one), token t takes g = dO_t + m_{t+1} and gives
//   dx = b g,  db = x g,  da = g h_{t-1},  m_t = a g,
// so that m runs through the maps (a, a dO) from the last token to the first,
// and h_{t-1} is walked again from the state saved at the tile's first token.
template <bool BF16, int FORM, int VEC>
__global__ __launch_bounds__(kNT) void linear_backward_seq(Lin p) {
  using G = Geo<VEC>;
  constexpr bool GB = BF16 && Form<FORM>::pre;
  __shared__ float2 tot[2][2][4][kLinChannels];
  const int tid = threadIdx.x, ct = tid % G::CT, s = tid / G::CT;
  const int n = blockIdx.x / p.nblk, blk = blockIdx.x - n * p.nblk;
  const int D = p.D, c0 = blk * kLinChannels + ct * VEC;
  const bool own = c0 < D;
  const int cc = own ? c0 : D - VEC;
  int lo = 0, hi = p.T;
  size_t row0 = (size_t)n * p.T;
  if (p.cu) {
    lo = clamp_offset(p.cu[n], p.T);
    hi = clamp_offset(p.cu[n + 1], p.T);
    row0 = 0;
  }
  const size_t ck0 = p.cu ? 0 : (size_t)n * ((p.T + kLinTile - 1) / kLinTile);
  float m[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) m[c] = p.dh_T ? p.dh_T[(size_t)n * D + cc + c] : 0.f;
  int par = 0;
  const int first = lo - lo % kLinTile;
  for (int t0 = hi > lo ? (hi - 1) - (hi - 1) % kLinTile : first - kLinTile; t0 >= first; t0 -= kLinTile, par ^= 1) {
    float hin[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c)
      hin[c] = t0 > lo ? p.ck[(ck0 + t0 / kLinTile) * D + cc + c] : p.h0 ? p.h0[(size_t)n * D + cc + c] : 0.f;
    float a[G::L][VEC], x[G::L][VEC], b[G::L][VEC], dO[G::L][VEC];
    const int ts = t0 + s * G::L;
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int t = ts + i, tc = t < lo ? lo : t >= hi ? hi - 1 : t;
      const size_t at = (row0 + tc) * D + cc;
      load_f<BF16>(x[i], p.x, at);
      load_f<GB>(a[i], p.a, at);
      if constexpr (!Form<FORM>::tied) load_f<GB>(b[i], p.b, at);
      load_f<BF16>(dO[i], p.dO, at);
      activate<FORM>(a[i], b[i]);
      if (t != tc) {
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          a[i][c] = 1.f;
          b[i][c] = x[i][c] = dO[i][c] = 0.f;
        }
      }
    }
    float A[VEC], U[VEC], Am[VEC], Um[VEC], h[VEC], mi[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      A[c] = 1.f;
      U[c] = Um[c] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        U[c] = __builtin_fmaf(a[i][c], U[c], b[i][c] * x[i][c]);
        A[c] *= a[i][c];
        const float *r = a[G::L - 1 - i], *d = dO[G::L - 1 - i];
        Um[c] = r[c] * (d[c] + Um[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) Am[c] = A[c];
    wave_scan<VEC, false>(A, U, tot[par][0], tid);
    wave_scan<VEC, true>(Am, Um, tot[par][1], tid);
    __syncthreads();
    enter<VEC, false>(h, hin, A, U, tot[par][0], tid);
    enter<VEC, true>(mi, m, Am, Um, tot[par][1], tid);
    float hp[G::L][VEC];
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        hp[i][c] = h[c];
        h[c] = __builtin_fmaf(a[i][c], h[c], b[i][c] * x[i][c]);
      }
    }
#pragma unroll
    for (int i = G::L - 1; i >= 0; --i) {
      const int t = ts + i;
      float dx[VEC], da[VEC], db[VEC];
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const float g = dO[i][c] + mi[c];
        mi[c] = a[i][c] * g;
        dx[c] = b[i][c] * g;
        db[c] = x[i][c] * g;
        da[c] = Form<FORM>::tied ? g * (hp[i][c] - x[i][c]) : g * hp[i][c];
      }
      if (own && t >= lo && t < hi) {
        const size_t at = (row0 + t) * D + c0;
        if constexpr (Form<FORM>::pre) {
          // through the activations: a' = -a (1 - a), b' = b (1 - b), the
          // complements again without a difference
          float pa[VEC], pb[VEC];
          load_f<GB>(pa, p.a, at);
          if constexpr (!Form<FORM>::tied) load_f<GB>(pb, p.b, at);
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            float y, z;
            split_sigmoid(pa[c], y, z);
            da[c] *= -y * z;
            if constexpr (!Form<FORM>::tied) {
              split_sigmoid(pb[c], y, z);
              db[c] *= y * z;
            }
          }
        }
        store_f<BF16>(p.dx, at, dx);
        store_f<GB>(p.da, at, da);
        if constexpr (!Form<FORM>::tied) store_f<GB>(p.db, at, db);
      }
    }
  }
  if (p.dh0 && own && s == 0) store_f<false>(p.dh0, (size_t)n * D + c0, m);
}

// One token: a thread per VEC channels of a row.
template <bool BF16, int FORM, int VEC>
__global__ __launch_bounds__(kNT) void linear_step(Lin p, size_t total) {
  constexpr bool GB = BF16 && Form<FORM>::pre;
  for (size_t i = ((size_t)blockIdx.x * kNT + threadIdx.x) * VEC; i < total; i += (size_t)gridDim.x * kNT * VEC) {
    float a[VEC], b[VEC], x[VEC], h[VEC];
    load_f<false>(h, p.h0, i);
    load_f<GB>(a, p.a, i);
    if constexpr (!Form<FORM>::tied) load_f<GB>(b, p.b, i);
    load_f<BF16>(x, p.x, i);
    activate<FORM>(a, b);
#pragma unroll
    for (int c = 0; c < VEC; ++c) h[c] = __builtin_fmaf(a[c], h[c], b[c] * x[c]);
    store_f<false>(p.h_T, i, h);
    store_f<BF16>(p.o, i, h);
  }
}

enum Op { kForward, kBackward, kStep };

template <bool BF16, int FORM, int VEC>
hipError_t launch_v(const LinearArgs &q, Op op, hipStream_t st) {
  Lin p{q.x, q.a, q.b, q.h0, q.o, q.h_T, q.ck, q.dO, q.dh_T, q.dx, q.da, q.db, q.dh0, q.cu, q.B, q.T, q.D, 0};
  p.nblk = (q.D + kLinChannels - 1) / kLinChannels;
  if (op == kStep) {
    const size_t total = (size_t)q.B * q.D, per = (size_t)kNT * VEC;
    const size_t wgs = (total + per - 1) / per;
    hipLaunchKernelGGL((linear_step<BF16, FORM, VEC>), dim3((unsigned)(wgs < 65536 ? wgs : 65536)), dim3(kNT), 0, st, p,
                       total);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((size_t)q.B * p.nblk));
  if (op == kForward)
    hipLaunchKernelGGL((linear_forward_seq<BF16, FORM, VEC>), grid, dim3(kNT), 0, st, p);
  else
    hipLaunchKernelGGL((linear_backward_seq<BF16, FORM, VEC>), grid, dim3(kNT), 0, st, p);
  return hipGetLastError();
}

template <bool BF16, int FORM>
hipError_t launch_f(const LinearArgs &q, Op op, hipStream_t st) {
  // four channels a thread where every row of every tensor is aligned to
  // their wide loads, else one
  uintptr_t at = 0;
  for (const void *p : {q.x, q.a, q.b, (const void *)q.h0, (const void *)q.o, (const void *)q.h_T, (const void *)q.ck,
                        q.dO, (const void *)q.dh_T, (const void *)q.dx, (const void *)q.da, (const void *)q.db,
                        (const void *)q.dh0})
    at |= reinterpret_cast<uintptr_t>(p);
  return q.D % 4 == 0 && (at & 15) == 0 ? launch_v<BF16, FORM, 4>(q, op, st) : launch_v<BF16, FORM, 1>(q, op, st);
}

template <bool BF16>
hipError_t launch_t(const LinearArgs &q, Op op, hipStream_t st) {
  switch (q.gates) {
    case GDN2_LINEAR_CHANNEL: return launch_f<BF16, GDN2_LINEAR_CHANNEL>(q, op, st);
    case GDN2_LINEAR_PREACT: return launch_f<BF16, GDN2_LINEAR_PREACT>(q, op, st);
    case GDN2_LINEAR_TIED: return launch_f<BF16, GDN2_LINEAR_TIED>(q, op, st);
    case GDN2_LINEAR_TIED_PREACT: return launch_f<BF16, GDN2_LINEAR_TIED_PREACT>(q, op, st);
  }
  return hipErrorInvalidValue;
}

hipError_t launch(const LinearArgs &q, Op op, hipStream_t st) {
  return q.bf16 ? launch_t<true>(q, op, st) : launch_t<false>(q, op, st);
}

}  // namespace

hipError_t launch_linear_forward(const LinearArgs &q, hipStream_t st) { return launch(q, kForward, st); }

hipError_t launch_linear_backward(const LinearArgs &q, hipStream_t st) {
  LinearArgs p = q;
  if (!p.ck) {  // the saved states again: a forward pass that writes nothing else
    p.ck = static_cast<float *>(p.workspace);
    LinearArgs f = p;
    f.o = nullptr;
    f.h_T = nullptr;
    const hipError_t e = launch(f, kForward, st);
    if (e != hipSuccess) return e;
  }
  return launch(p, kBackward, st);
}

hipError_t launch_linear_step(const LinearArgs &q, hipStream_t st) { return launch(q, kStep, st); }

}  // namespace gdn2
