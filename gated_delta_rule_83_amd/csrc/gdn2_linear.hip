// gdn2_linear.hip -- the gated linear recurrence h_t = a_t h_{t-1} + b_t x_t,
// channel by channel, its gradients, and its single-token step.
//
// A token is the map h -> a h + u (u = b x); maps compose:
//   (a2, u2) after (a1, u1) = (a2 a1, a2 u1 + u2).
// A workgroup of 256 threads owns 128 channels and holds 64 tokens of them in
// registers: VEC channels (one wide load) by L = 64 / slots consecutive tokens
// a thread. It composes each thread's tokens, scans the threads' maps (lane
// shuffles inside a wave, LDS across waves), and walks its tokens again from
// the state that enters them. Everything between the loads
// and the one rounding of an output is fp32.
#include "gdn2_linear.hpp"
#include "gdn2_vec.hpp"

#include "gdn2.h"

#include <initializer_list>

namespace gdn2 {

namespace {

constexpr int kNT = 256, kTeams = kNT / kLinChannels;  // threads of a workgroup, and of them per channel
constexpr int kStepNT = 256;

// Token tensors are read with nontemporal loads (load_raw). A pass over the
// bytes of the forward in tiles, bf16, 32768 x 2048: with tiles of 64 channels
// 5.2 TB/s without them and 5.6 to 6.2 with them, with tiles of 128 channels
// (rows of 256 bytes) 6.3 TB/s. (In the whole kernel 64 channels by 128 tokens
// took 8% longer than 128 by 64, 256 by 32 took 4%, and 512 threads with 128
// by 128 took 35%.)

// 1 / (1 + e^x). e^x may be infinite (0). EXACT (fp32 pre-activations): the
// reciprocal's error of one step taken out by a Newton step, x above 87 as 87
// (1.6e-38); a bf16 pre-activation is itself off by 2^-9 of its size.
template <bool EXACT> __device__ __forceinline__ float low_sigmoid(float x) {
  if constexpr (EXACT) x = x > 87.f ? 87.f : x;
  const float d = 1.f + __builtin_amdgcn_exp2f(x * 1.44269504088896341f), r = __builtin_amdgcn_rcpf(d);
  return EXACT ? __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r) : r;
}

template <int FORM> struct Form {
  static constexpr bool pre = FORM == GDN2_LINEAR_PREACT || FORM == GDN2_LINEAR_TIED_PREACT;
  static constexpr bool tied = FORM == GDN2_LINEAR_TIED || FORM == GDN2_LINEAR_TIED_PREACT;
};

// A value's gates from what was loaded: decay a, input gate b. 1 - a comes
// from its own sigmoid, so that it keeps its relative accuracy as a nears 1;
// a is then off by at most 2^-24.
template <int FORM, bool EXACT> __device__ __forceinline__ void activate(float &a, float &b) {
  if constexpr (FORM == GDN2_LINEAR_PREACT) {
    a = low_sigmoid<EXACT>(a);
    b = low_sigmoid<EXACT>(-b);
  } else if constexpr (FORM == GDN2_LINEAR_TIED_PREACT) {
    b = low_sigmoid<EXACT>(-a);
    a = 1.f - b;
  } else if constexpr (FORM == GDN2_LINEAR_TIED) {
    b = 1.f - a;
  }
}

// A sigmoid p = 1 / (1 + e^x) and its complement q in one word v: the smaller of
// the two, e^-|x| / (1 + e^-|x|), with x's sign, so p where that is at most 1/2
// and -q above. Both come back, and p q, without a difference that loses digits:
// a gradient through a nearly closed or open gate keeps its relative accuracy.
// (What is added is the smallest normal number: v is never 0, which has no side.)
constexpr float kNoSlope = 0x1p-126f;
template <bool EXACT> __device__ __forceinline__ float pack_pair(float x) {
  const float e = __builtin_amdgcn_exp2f(__builtin_fabsf(x) * -1.44269504088896341f), d = 1.f + e;
  float r = __builtin_amdgcn_rcpf(d);
  if constexpr (EXACT) r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
  return __builtin_copysignf(__builtin_fmaf(e, r, kNoSlope), x);
}
__device__ __forceinline__ float pair_p(float v) { return v - __builtin_floorf(v); }
__device__ __forceinline__ float pair_q(float v) { return __builtin_ceilf(v) - v; }
__device__ __forceinline__ float pair_pq(float v) { return __builtin_fmaf(-v, v, __builtin_fabsf(v)); }

// A token's gates as the backward keeps them, one word each: fp32 gates
// themselves, pre-activations' as pairs.
template <int FORM, bool EXACT> struct Gates {
  static __device__ __forceinline__ void pack(float &a, float &b) {
    if constexpr (Form<FORM>::pre) {
      a = pack_pair<EXACT>(a);
      if constexpr (!Form<FORM>::tied) b = pack_pair<EXACT>(-b);
    }
  }
  static __device__ __forceinline__ void unpack(float va, float vb, float &a, float &b) {
    a = Form<FORM>::pre ? pair_p(va) : va;
    if constexpr (Form<FORM>::tied) b = Form<FORM>::pre ? pair_q(va) : 1.f - va;
    else b = Form<FORM>::pre ? pair_p(vb) : vb;
  }
  // va of a token that passes the state on (a = 1)
  static __device__ __forceinline__ float none() { return Form<FORM>::pre ? -kNoSlope : 1.f; }
};

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

// Geometry of a thread: ct-th group of VEC channels, s-th slot of L tokens;
// WS slots a wave, in scans of PARTS parts of whole waves.
template <int VEC> struct Geo {
  static constexpr int CT = kLinChannels / VEC, NS = kNT / CT, L = kLinTile / NS;
  static constexpr int PART = CT < 64 ? 64 : CT, WS = PART / CT, PARTS = kNT / PART;
};

// A map that takes nothing from what lies before it, not even a NaN or an
// infinity: that is how a sequence of a packed batch starts. No product of
// decays is this value; one that is 0 passes a NaN on.
constexpr float kCut = -__builtin_huge_valf();

// (A, U) := (a, u) after (A, U). CUT: either may be a cut.
template <bool CUT> __device__ __forceinline__ void after(float a, float u, float &A, float &U) {
  if (CUT && a == kCut) {
    A = kCut;
    U = u;
  } else {
    U = __builtin_fmaf(a, U, u);
    A = CUT && A == kCut ? A : A * a;
  }
}
template <bool CUT> __device__ __forceinline__ float apply(float a, float u, float h) {
  return CUT && a == kCut ? u : __builtin_fmaf(a, h, u);
}

// Where a tile's token tensors lie: the tile's first value, the bytes from a
// token to the next, and this lane's offset from the tile's first value.
template <bool BF16> struct Span {
  size_t first;
  uint32_t row, lane;
  __device__ __forceinline__ Span(size_t at, int D, uint32_t lane_at) {
    constexpr uint32_t es = sizeof(typename Elem<BF16>::T);
    first = at * es;
    row = (uint32_t)D * es;
    lane = lane_at * es;
  }
  template <int N> __device__ __forceinline__ Raw<BF16, N> load(const void *p, int i) const {
    return load_raw<BF16, N>(static_cast<const char *>(p) + first + (size_t)((uint64_t)row * i), lane);
  }
  template <int N> __device__ __forceinline__ void store(void *p, int i, const float (&f)[N]) const {
    store_at<BF16>(static_cast<char *>(p) + first + (size_t)((uint64_t)row * i) + lane, f);
  }
};

// Scan of the threads' maps (A, U) in token order (or, REV, from the last
// token to the first): on return (A, U) is the map of all earlier threads of
// this part, and tot[w] in LDS the whole map of part w. A part is one slot
// (VEC = 1), or a wave of two, whose halves swap their maps in registers.
template <int VEC, bool REV, bool CUT>
__device__ __forceinline__ void wave_scan(float (&A)[VEC], float (&U)[VEC], float2 (*tot)[kLinChannels], int tid) {
  using G = Geo<VEC>;
  static_assert(G::WS == 1 || (G::WS == 2 && G::CT == 32), "slots of a part");
  const int w = tid / G::PART, ct = tid % G::CT;
  if constexpr (G::WS == 1) {
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      tot[w][ct * VEC + c] = float2{A[c], U[c]};
      A[c] = 1.f;
      U[c] = 0.f;
    }
  } else {
    const bool later = ((tid & 32) != 0) != REV;  // this half comes after the other one
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      // [0]: the lower half's value in both halves, [1]: the upper half's
      const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(A[c]), __float_as_uint(A[c]), false, false);
      const auto u = __builtin_amdgcn_permlane32_swap(__float_as_uint(U[c]), __float_as_uint(U[c]), false, false);
      const float a0 = __uint_as_float(a[REV ? 1 : 0]), u0 = __uint_as_float(u[REV ? 1 : 0]);
      A[c] = a0;
      U[c] = u0;
      after<CUT>(__uint_as_float(a[REV ? 0 : 1]), __uint_as_float(u[REV ? 0 : 1]), A[c], U[c]);
      if (!later) tot[w][ct * VEC + c] = float2{A[c], U[c]};
      A[c] = later ? a0 : 1.f;
      U[c] = later ? u0 : 0.f;
    }
  }
}

// The value entering this thread's tokens and the value leaving the tile,
// from the value entering the tile (carry, replaced by the leaving one).
template <int VEC, bool REV, bool CUT>
__device__ __forceinline__ void enter(float (&in)[VEC], float (&carry)[VEC], const float (&A)[VEC],
                                      const float (&U)[VEC], const float2 (*tot)[kLinChannels], int tid) {
  using G = Geo<VEC>;
  const int w = tid / G::PART, ct = tid % G::CT;
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    float h = carry[c], mine = h;
#pragma unroll
    for (int i = 0; i < G::PARTS; ++i) {
      const int j = REV ? G::PARTS - 1 - i : i;
      if (j == w) mine = h;
      const float2 t = tot[j][ct * VEC + c];
      h = apply<CUT>(t.x, t.y, h);
    }
    in[c] = apply<CUT>(A[c], U[c], mine);
    carry[c] = h;
  }
}

// ------------------------------------------------------------------ tiles in parallel
// The tiles of one chain (a sequence's, or the packed axis', and 128 channels)
// run at once, each read from memory once. A workgroup takes its chain's next
// tile by a ticket, so that every tile it waits for was taken before it and is
// running or done: no wait is endless. (A ticket per chain: one counter for all
// of them hands out a tile every 15 ns, which bound the whole kernel.) It
// publishes its tile's map, and finds the value entering the tile from
//   the maps of the tiles before it in its group of kGroup tiles, composed,
//   applied to the value that left the group before (published by that
//   group's last tile): the same sums in the same order whatever the timing.
// Each published word validates itself (a map's two floats in 64 bits, a
// value in 32; all bits set: not there yet; NaN published as the quiet NaN),
// so relaxed agent-scope accesses suffice: no fence writes a cache back.
constexpr int kGroup = 8;  // 16: each tile reads twice as many maps, 1 to 4% slower
constexpr int kTicketWords = 16;
constexpr int kDies = 8, kSpread = 2048;  // dies; the largest grid that takes the chains in turn
constexpr int kSpins = 1 << 24;  // a wait given up after this many looks yields NaN

struct Chain {
  uint32_t *ticket;  // [chain], kTicketWords apart
  uint64_t *map;    // [tile][chain][kLinChannels]
  uint32_t *value;  // [group][chain][kLinChannels]
  int chains, tiles;
  int by_die;  // workgroups that take one chain in eights, the first of the grid (take_tile)
};

__device__ __forceinline__ uint32_t word(float f) { return f != f ? 0x7fc00000u : __float_as_uint(f); }

// Tile of this workgroup: its index k along the walk and its chain.
__device__ __forceinline__ void take_tile(const Chain &ch, int *slot, int tid, int &k, int &chain) {
  // Workgroups go round the eight dies in turn. In a large grid eight in a row
  // take one chain, so that a tile's neighbours in channels mostly run on its own
  // die and find the lines they share in its L2: bf16 forward 158 -> 150 us (B8
  // T4096 D2048, channel), 236 -> 206 (B1 T65536 D2048), backward at rows that are
  // no multiple of a line 135 -> 116 (B4 T8192 D1004). A small one, where the
  // chain's own steps count, takes the chains in turn: 13 us against 15 (B1 T2048
  // D2048), backward 53 against 57 (B16 T512 D2048). They meet at 2048 workgroups.
  const int b = blockIdx.x;
  chain = (b < ch.by_die ? b / kDies : b - ch.by_die) % ch.chains;
  k = 0;
  if (ch.tiles > 1) {
    if (tid == 0)  // the tickets start at 2^32 - 1
      *slot = (int)(__hip_atomic_fetch_add(ch.ticket + (size_t)chain * kTicketWords, 1u, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT) + 1u);
    __syncthreads();
    k = __builtin_amdgcn_readfirstlane(*slot);
  }
}

// The value entering tile k of its chain, for this thread's channel in the
// first kLinChannels threads, from the tiles' published maps; own: this tile's
// map. Publishes both. Every thread of the workgroup calls it. start: the value
// entering the chain, in its first tile (0 in others). That tile publishes the
// value leaving it as a map that takes nothing, so that no other one reads where
// start lies: the chain's last value may be written there.
template <bool CUT>
__device__ __forceinline__ float link(const Chain &ch, int k, int chain, float2 own, float start,
                                      float2 (*maps)[kLinChannels], int tid) {
  const int lane = tid % kLinChannels, w = tid / kLinChannels, in = k % kGroup;
  if (ch.tiles == 1) return start;
  if (k == 0) own = float2{CUT ? kCut : 0.f, apply<CUT>(own.x, own.y, start)};
  if (w == 0 && in != kGroup - 1 && k != ch.tiles - 1)
    __hip_atomic_store(ch.map + ((size_t)k * ch.chains + chain) * kLinChannels + lane,
                       (uint64_t)word(own.x) | (uint64_t)word(own.y) << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t *before = ch.value + ((size_t)(k / kGroup - 1) * ch.chains + chain) * kLinChannels + lane;
  uint32_t p = ~0u;
  auto look = [&] { p = __hip_atomic_load(before, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  if (w == 0 && k >= kGroup) look();  // mostly there before the maps are
  uint64_t v[kGroup / kTeams];
  const uint64_t *at = ch.map + ((size_t)(k - in + w) * ch.chains + chain) * kLinChannels + lane;
  for (int spin = 0; spin < kSpins; ++spin) {
    bool ready = true;
#pragma unroll
    for (int j = 0; j < kGroup / kTeams; ++j) {
      v[j] = 0;
      if (kTeams * j + w < in)
        v[j] = __hip_atomic_load(at + (size_t)kTeams * j * ch.chains * kLinChannels, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
      ready = ready && v[j] != ~(uint64_t)0;
    }
    if (ready) break;
    __builtin_amdgcn_s_sleep(1);
  }
#pragma unroll
  for (int j = 0; j < kGroup / kTeams; ++j)
    maps[kTeams * j + w][lane] = float2{__uint_as_float((uint32_t)v[j]), __uint_as_float((uint32_t)(v[j] >> 32))};
  __syncthreads();
  if (w != 0) return 0.f;
  float A = 1.f, U = 0.f;
  for (int j = 0; j < in; ++j) after<CUT>(maps[j][lane].x, maps[j][lane].y, A, U);
  float h = start;
  if (k >= kGroup) {
    for (int spin = 0; spin < kSpins && p == ~0u; ++spin) {
      __builtin_amdgcn_s_sleep(1);
      look();
    }
    h = __uint_as_float(p);  // all bits set is a NaN
  }
  h = apply<CUT>(A, U, h);
  if (in == kGroup - 1 && k != ch.tiles - 1)
    __hip_atomic_store(ch.value + ((size_t)(k / kGroup) * ch.chains + chain) * kLinChannels + lane,
                       word(apply<CUT>(own.x, own.y, h)), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return h;
}

// A tile's map from its parts', for one channel.
template <int PARTS, bool REV, bool CUT>
__device__ __forceinline__ float2 tile_map(const float2 (*tot)[kLinChannels], int channel) {
  float A = 1.f, U = 0.f;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const float2 t = tot[REV ? PARTS - 1 - i : i][channel];
    after<CUT>(t.x, t.y, A, U);
  }
  return float2{A, U};
}

// Which sequence starts and which ends at each token of a packed tile (-1: none).
struct Edges {
  int start[kLinTile], end[kLinTile];
};

// Bit i: whether token s L + i of the tile has such an edge.
template <int L> __device__ __forceinline__ uint32_t edge_bits(const int *at, int s) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < L; ++i) m |= at[s * L + i] >= 0 ? 1u << i : 0u;
  return m;
}

__device__ __forceinline__ void find_edges(Edges &e, const Lin &p, int t0, int tid) {
  if (tid < kLinTile) e.start[tid] = e.end[tid] = -1;
  // the first sequence that may reach into the tile, to within kNT
  int lo = 0, hi = p.B;
  while (hi - lo > kNT) {
    const int mid = lo + (hi - lo) / 2;
    if (clamp_offset(p.cu[mid], p.T) <= t0) lo = mid;
    else hi = mid;
  }
  __syncthreads();
  for (int n = lo + tid; n < p.B; n += kNT) {
    const int b = clamp_offset(p.cu[n], p.T), f = clamp_offset(p.cu[n + 1], p.T);
    if (b >= t0 + kLinTile) break;
    if (b >= f) continue;
    if (b >= t0) e.start[b - t0] = n;
    if (f > t0 && f <= t0 + kLinTile) e.end[f - 1 - t0] = n;
  }
  __syncthreads();
}

template <bool BF16, int FORM, int VEC, bool PACKED>
__global__ __launch_bounds__(kNT, VEC == 4 ? 4 : 1) void linear_forward_chain(Lin p, Chain ch) {
  using G = Geo<VEC>;
  constexpr bool GB = BF16 && Form<FORM>::pre;
  __shared__ float2 tot[G::PARTS][kLinChannels], maps[kGroup][kLinChannels];
  __shared__ float entering[kLinChannels];
  __shared__ Edges edges[1];
  __shared__ int slot;
  const int tid = threadIdx.x, lane = tid % kLinChannels, ct = tid % G::CT, s = tid / G::CT;
  int k, chain;
  take_tile(ch, &slot, tid, k, chain);
  const int n = PACKED ? 0 : chain / p.nblk, blk = chain - n * p.nblk;
  const int D = p.D, c0 = blk * kLinChannels + ct * VEC;
  const bool own = c0 < D;
  const int cc = own ? c0 : D - VEC, t0 = k * kLinTile, ts = t0 + s * G::L;
  int lo = 0, hi = p.T;
  if constexpr (PACKED) {
    lo = clamp_offset(p.cu[0], p.T);
    hi = clamp_offset(p.cu[p.B], p.T);
  }
  const size_t row0 = PACKED ? 0 : (size_t)n * p.T, ck0 = PACKED ? 0 : (size_t)n * ch.tiles;

  const size_t first = (row0 + t0) * D + blk * kLinChannels;
  const uint32_t lane_at = (uint32_t)(s * G::L) * D + (cc - blk * kLinChannels);
  const Span<BF16> sx(first, D, lane_at);
  const Span<GB> sg(first, D, lane_at);
  const bool ragged = t0 < lo || t0 + kLinTile > hi;
  Raw<BF16, VEC> xr[G::L];
  Raw<GB, VEC> ar[G::L], br[G::L];
  auto load = [&](int i) {
    xr[i] = sx.template load<VEC>(p.x, i);
    ar[i] = sg.template load<VEC>(p.a, i);
    if constexpr (!Form<FORM>::tied) br[i] = sg.template load<VEC>(p.b, i);
  };
  if (!ragged) {
#pragma unroll
    for (int i = 0; i < G::L; ++i) load(i);
  } else {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      xr[i] = {};
      ar[i] = br[i] = {};
      if (ts + i < p.T) load(i);
    }
  }
  uint32_t starts = 0, ends = 0;  // of this thread's tokens
  if constexpr (PACKED) {
    find_edges(edges[0], p, t0, tid);
    starts = edge_bits<G::L>(edges[0].start, s);
    ends = edge_bits<G::L>(edges[0].end, s);
  }
  float a[G::L][VEC], u[G::L][VEC];
#pragma unroll
  for (int i = 0; i < G::L; ++i) {
    const int t = ts + i;
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float av = ar[i][c], bv = 0.f;
      if constexpr (!Form<FORM>::tied) bv = br[i][c];
      activate<FORM, !BF16>(av, bv);
      u[i][c] = bv * xr[i][c];
      a[i][c] = av;
    }
    if (ragged && (t < lo || t >= hi)) {  // no token: the identity map
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        u[i][c] = 0.f;
        a[i][c] = 1.f;
      }
    }
  }
  float A[VEC], U[VEC], h[VEC], carry[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    A[c] = 1.f;
    U[c] = 0.f;
  }
  if (!PACKED || !starts) {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) after<false>(a[i][c], u[i][c], A[c], U[c]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      if (starts >> i & 1) {  // a sequence starts: its own state, and a cut
        const int q = edges[0].start[s * G::L + i];
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          if (p.h0) u[i][c] = __builtin_fmaf(a[i][c], p.h0[(size_t)q * D + cc + c], u[i][c]);
          U[c] = u[i][c];
        }
      } else {
#pragma unroll
        for (int c = 0; c < VEC; ++c) U[c] = __builtin_fmaf(a[i][c], U[c], u[i][c]);
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) A[c] = kCut;
  }
  wave_scan<VEC, false, PACKED>(A, U, tot, tid);
  __syncthreads();
  {
    const int c = blk * kLinChannels + lane;
    const float start = !PACKED && k == 0 && p.h0 && c < D && tid < kLinChannels ? p.h0[(size_t)n * D + c] : 0.f;
    const float in = link<PACKED>(ch, k, chain, tile_map<G::PARTS, false, PACKED>(tot, lane), start, maps, tid);
    if (tid < kLinChannels) {
      entering[lane] = in;
      if (p.ck && k > 0 && c < D) p.ck[(ck0 + k) * D + c] = in;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < VEC; ++c) carry[c] = entering[ct * VEC + c];
  enter<VEC, false, PACKED>(h, carry, A, U, tot, tid);
  if (!PACKED || !(starts | ends)) {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int t = ts + i;
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = __builtin_fmaf(a[i][c], h[c], u[i][c]);
      if (own && p.o && (!ragged || (t >= lo && t < hi))) sx.store(p.o, i, h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int t = ts + i;
      const bool cut = starts >> i & 1;
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = cut ? u[i][c] : __builtin_fmaf(a[i][c], h[c], u[i][c]);
      if (own && t >= lo && t < hi) {
        if (p.o) sx.store(p.o, i, h);
        if ((ends >> i & 1) && p.h_T) store_f<false>(p.h_T, (size_t)edges[0].end[s * G::L + i] * D + c0, h);
      }
    }
  }
  if (!PACKED && p.h_T && k == ch.tiles - 1 && own && s == 0) store_f<false>(p.h_T, (size_t)n * D + c0, carry);
}

// The gradients, tile by tile from the last one: the adjoint is chained, the
// states come from the saved ones. Two waves a SIMD: fp32 with untied gates and
// packed single values would take a few registers past the half of them (B4
// T4096 D2048 fp32 pre-activations 229 us instead of 196, packed 16384 x 1001
// bf16 pre-activations 150 instead of 101).
template <bool BF16, int FORM, int VEC, bool PACKED>
__global__ __launch_bounds__(kNT, 2) void linear_backward_chain(Lin p, Chain ch) {
  using G = Geo<VEC>;
  constexpr bool GB = BF16 && Form<FORM>::pre;
  __shared__ float2 tot[2][G::PARTS][kLinChannels], maps[kGroup][kLinChannels];
  __shared__ float entering[kLinChannels];
  __shared__ Edges edges[1];
  __shared__ float last[PACKED ? kLinTile : 1][kLinChannels];
  __shared__ int slot;
  const int tid = threadIdx.x, lane = tid % kLinChannels, ct = tid % G::CT, s = tid / G::CT;
  int k, chain;
  take_tile(ch, &slot, tid, k, chain);
  const int n = PACKED ? 0 : chain / p.nblk, blk = chain - n * p.nblk;
  const int D = p.D, c0 = blk * kLinChannels + ct * VEC;
  const bool own = c0 < D;
  const int tile = ch.tiles - 1 - k;
  const int cc = own ? c0 : D - VEC, t0 = tile * kLinTile, ts = t0 + s * G::L;
  int lo = 0, hi = p.T;
  if constexpr (PACKED) {
    lo = clamp_offset(p.cu[0], p.T);
    hi = clamp_offset(p.cu[p.B], p.T);
  }
  const size_t row0 = PACKED ? 0 : (size_t)n * p.T, ck0 = PACKED ? 0 : (size_t)n * ch.tiles;

  using GT = Gates<FORM, !BF16>;
  Raw<BF16, VEC> x[G::L], dr[G::L];
  float va[G::L][VEC], vb[G::L][VEC], hin[VEC];
  const size_t first = (row0 + t0) * D + blk * kLinChannels;
  const uint32_t lane_at = (uint32_t)(s * G::L) * D + (cc - blk * kLinChannels);
  const Span<BF16> sx(first, D, lane_at);
  const Span<GB> sg(first, D, lane_at);
  const bool ragged = t0 < lo || t0 + kLinTile > hi;
  {
    Raw<GB, VEC> ar[G::L], br[G::L];
    auto load = [&](int i) {
      x[i] = sx.template load<VEC>(p.x, i);
      ar[i] = sg.template load<VEC>(p.a, i);
      if constexpr (!Form<FORM>::tied) br[i] = sg.template load<VEC>(p.b, i);
      dr[i] = sx.template load<VEC>(p.dO, i);
    };
    if (!ragged) {
#pragma unroll
      for (int i = 0; i < G::L; ++i) load(i);
    } else {
#pragma unroll
      for (int i = 0; i < G::L; ++i) {
        x[i] = dr[i] = {};
        ar[i] = br[i] = {};
        if (ts + i < p.T) load(i);
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c)
      hin[c] = tile > 0 ? p.ck[(ck0 + tile) * D + cc + c] : !PACKED && p.h0 ? p.h0[(size_t)n * D + cc + c] : 0.f;
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        va[i][c] = ar[i][c];
        vb[i][c] = 0.f;
        if constexpr (!Form<FORM>::tied) vb[i][c] = br[i][c];
        GT::pack(va[i][c], vb[i][c]);
      }
      if (ragged && (ts + i < lo || ts + i >= hi)) {  // no token: the identity map
        x[i] = dr[i] = {};
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          va[i][c] = GT::none();
          vb[i][c] = 0.f;
        }
      }
    }
  }
  // a packed sequence's last token takes its state's gradient too: read before
  // anything is published (dh0 may be dh_T) and kept where only this thread looks
  uint32_t starts = 0, ends = 0;
  if constexpr (PACKED) {
    find_edges(edges[0], p, t0, tid);
    starts = edge_bits<G::L>(edges[0].start, s);
    ends = edge_bits<G::L>(edges[0].end, s);
    for (uint32_t m = ends; m; m &= m - 1) {
      const int at = s * G::L + __builtin_ctz(m);
#pragma unroll
      for (int c = 0; c < VEC; ++c)
        last[at][ct * VEC + c] = p.dh_T ? p.dh_T[(size_t)edges[0].end[at] * D + cc + c] : 0.f;
    }
  }
  // between the passes over the tokens: what is unpacked for one pass is not
  // kept for the next (256 + 97 registers otherwise, bf16 pre-activations)
  auto hold = [&] {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      pin_regs(va[i]);
      if constexpr (!Form<FORM>::tied) pin_regs(vb[i]);
      if constexpr (sizeof(x[i]) % 4 == 0) {
        pin_regs(x[i].v);
        pin_regs(dr[i].v);
      }
    }
  };
  float A[VEC], U[VEC], Am[VEC], Um[VEC], h[VEC], mi[VEC], m[VEC];
#pragma unroll
  for (int c = 0; c < VEC; ++c) {
    A[c] = Am[c] = 1.f;
    U[c] = Um[c] = 0.f;
  }
  if (!PACKED || !(starts | ends)) {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int j = G::L - 1 - i;
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float a, b, am, bm;
        GT::unpack(va[i][c], vb[i][c], a, b);
        GT::unpack(va[j][c], vb[j][c], am, bm);
        U[c] = __builtin_fmaf(a, U[c], b * x[i][c]);
        A[c] *= a;
        Um[c] = am * (dr[j][c] + Um[c]);
      }
      // packed single values: unpacking that runs ahead spills (fp32, 16384 x 1001: 159 us instead of 134)
      if constexpr (PACKED && VEC == 1 && Form<FORM>::pre) __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) Am[c] = A[c];
  } else {
#pragma unroll
    for (int i = 0; i < G::L; ++i) {
      const int j = G::L - 1 - i;
      const bool first = starts >> i & 1, cut = ends >> j & 1;
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        float a, b, am, bm;
        GT::unpack(va[i][c], vb[i][c], a, b);
        GT::unpack(va[j][c], vb[j][c], am, bm);
        const float from = first ? (p.h0 ? p.h0[(size_t)edges[0].start[s * G::L + i] * D + cc + c] : 0.f) : U[c];
        U[c] = __builtin_fmaf(a, from, b * x[i][c]);
        A[c] *= a;
        Um[c] = am * (dr[j][c] + (cut ? last[s * G::L + j][ct * VEC + c] : Um[c]));
      }
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      Am[c] = ends ? kCut : A[c];
      A[c] = starts ? kCut : A[c];
    }
  }
  hold();
  wave_scan<VEC, false, PACKED>(A, U, tot[0], tid);
  wave_scan<VEC, true, PACKED>(Am, Um, tot[1], tid);
  __syncthreads();
  {
    const int c = blk * kLinChannels + lane;
    const float start = !PACKED && k == 0 && p.dh_T && c < D && tid < kLinChannels ? p.dh_T[(size_t)n * D + c] : 0.f;
    const float in = link<PACKED>(ch, k, chain, tile_map<G::PARTS, true, PACKED>(tot[1], lane), start, maps, tid);
    if (tid < kLinChannels) entering[lane] = in;
  }
  enter<VEC, false, PACKED>(h, hin, A, U, tot[0], tid);
  float hp[G::L][VEC];
#pragma unroll
  for (int i = 0; i < G::L; ++i) {
    if (PACKED && (starts >> i & 1)) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) h[c] = p.h0 ? p.h0[(size_t)edges[0].start[s * G::L + i] * D + cc + c] : 0.f;
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float a, b;
      GT::unpack(va[i][c], vb[i][c], a, b);
      hp[i][c] = h[c];
      h[c] = __builtin_fmaf(a, h[c], b * x[i][c]);
    }
  }
  hold();
  __syncthreads();
#pragma unroll
  for (int c = 0; c < VEC; ++c) m[c] = entering[ct * VEC + c];
  enter<VEC, true, PACKED>(mi, m, Am, Um, tot[1], tid);
#pragma unroll
  for (int i = G::L - 1; i >= 0; --i) {
    const int t = ts + i;
    float dx[VEC], da[VEC], db[VEC];
    if (PACKED && (ends >> i & 1)) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) mi[c] = last[s * G::L + i][ct * VEC + c];
    }
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      float a, b;
      GT::unpack(va[i][c], vb[i][c], a, b);
      const float g = dr[i][c] + mi[c], xv = x[i][c];
      mi[c] = a * g;
      dx[c] = b * g;
      db[c] = xv * g;
      da[c] = Form<FORM>::tied ? g * (hp[i][c] - xv) : g * hp[i][c];
      if constexpr (Form<FORM>::pre) {  // through the activations: a' = -a (1 - a), b' = b (1 - b)
        da[c] *= -pair_pq(va[i][c]);
        if constexpr (!Form<FORM>::tied) db[c] *= pair_pq(vb[i][c]);
      }
    }
    if (own && (!ragged || t < p.T)) {
      if (PACKED && ragged && (t < lo || t >= hi)) {  // no sequence's token: no gradient
#pragma unroll
        for (int c = 0; c < VEC; ++c) dx[c] = da[c] = db[c] = 0.f;
      }
      sx.store(p.dx, i, dx);
      sg.store(p.da, i, da);
      if constexpr (!Form<FORM>::tied) sg.store(p.db, i, db);
      if (PACKED && (starts >> i & 1) && p.dh0)
        store_f<false>(p.dh0, (size_t)edges[0].start[s * G::L + i] * D + c0, mi);
    }
  }
  if (!PACKED && p.dh0 && tile == 0 && own && s == 0) store_f<false>(p.dh0, (size_t)n * D + c0, m);
}

// Channels of a state that a workgroup passes on at a time, and such pieces of a state.
constexpr int kPass = 4096;
__host__ __device__ inline uint32_t pass_pieces(int D) { return (uint32_t)(D + kPass - 1) / kPass; }

// Before a chained launch: the words not published yet, and what needs no
// token: the states of empty sequences pass through (all of them without cu).
__global__ __launch_bounds__(kNT) void chain_prepare(uint4 *words, size_t count, const int32_t *cu, int B, int T, int D,
                                                     const float *from, float *to) {
  const size_t me = (size_t)blockIdx.x * kNT + threadIdx.x;
  for (size_t i = me; i < count; i += (size_t)gridDim.x * kNT) words[i] = uint4{~0u, ~0u, ~0u, ~0u};
  if (!to) return;
  const uint32_t per = pass_pieces(D);
  for (size_t i = blockIdx.x; i < (size_t)B * per; i += gridDim.x) {
    const int n = (int)(i / per), c0 = (int)(i - (size_t)n * per) * kPass;
    if (cu && clamp_offset(cu[n + 1], T) > clamp_offset(cu[n], T)) continue;
    const int end = c0 + kPass < D ? c0 + kPass : D;
    for (int c = c0 + threadIdx.x; c < end; c += kNT) to[(size_t)n * D + c] = from ? from[(size_t)n * D + c] : 0.f;
  }
}

// One token: a thread per VEC channels of a row.
template <bool BF16, int FORM, int VEC>
__global__ __launch_bounds__(kStepNT) void linear_step(Lin p, size_t total) {
  constexpr bool GB = BF16 && Form<FORM>::pre;
  for (size_t i = ((size_t)blockIdx.x * kStepNT + threadIdx.x) * VEC; i < total; i += (size_t)gridDim.x * kStepNT * VEC) {
    float a[VEC], b[VEC], x[VEC], h[VEC];
    load_f<false>(h, p.h0, i);
    load_f<GB>(a, p.a, i);
    if constexpr (!Form<FORM>::tied) load_f<GB>(b, p.b, i);
    load_f<BF16>(x, p.x, i);
#pragma unroll
    for (int c = 0; c < VEC; ++c) {
      activate<FORM, !BF16>(a[c], b[c]);
      h[c] = __builtin_fmaf(a[c], h[c], b[c] * x[c]);
    }
    store_f<false>(p.h_T, i, h);
    store_f<BF16>(p.o, i, h);
  }
}

enum Op { kForward, kBackward, kStep };

// Bytes of a chained launch's words: the tickets, the maps, the values.
size_t chain_bytes(int chains, int tiles) {
  if (tiles <= 1) return 0;
  return (size_t)chains * (kTicketWords * 4 + (size_t)tiles * kLinChannels * 8 +
                           (size_t)((tiles + kGroup - 1) / kGroup) * kLinChannels * 4);
}

template <bool BF16, int FORM, int VEC>
hipError_t launch_v(const LinearArgs &q, Op op, hipStream_t st) {
  Lin p{q.x, q.a, q.b, q.h0, q.o, q.h_T, q.ck, q.dO, q.dh_T, q.dx, q.da, q.db, q.dh0, q.cu, q.B, q.T, q.D, 0};
  p.nblk = (q.D + kLinChannels - 1) / kLinChannels;
  if (op == kStep) {
    const size_t total = (size_t)q.B * q.D, per = (size_t)kStepNT * VEC;
    const size_t wgs = (total + per - 1) / per;
    hipLaunchKernelGGL((linear_step<BF16, FORM, VEC>), dim3((unsigned)(wgs < 65536 ? wgs : 65536)), dim3(kStepNT), 0, st, p,
                       total);
    return hipGetLastError();
  }
  Chain ch{};
  ch.chains = (q.cu ? 1 : q.B) * p.nblk;
  ch.tiles = (q.T + kLinTile - 1) / kLinTile;
  const size_t bytes = chain_bytes(ch.chains, ch.tiles);
  if (bytes) {
    ch.ticket = static_cast<uint32_t *>(q.workspace);
    ch.map = reinterpret_cast<uint64_t *>(ch.ticket + (size_t)ch.chains * kTicketWords);
    ch.value = reinterpret_cast<uint32_t *>(ch.map + (size_t)ch.tiles * ch.chains * kLinChannels);
  }
  const float *from = op == kForward ? q.h0 : q.dh_T;
  float *to = !q.cu && ch.tiles ? nullptr : op == kForward ? q.h_T : q.dh0;
  if (bytes || to) {
    // enough workgroups for the words and for the states (64 tokens among 4096
    // sequences of 4096 channels: 16 ms with one)
    const size_t count = bytes / 16, wgs = (count + kNT - 1) / kNT, pass = to ? (size_t)q.B * pass_pieces(q.D) : 0;
    const size_t most = wgs > pass ? wgs : pass, grid = most < 1 ? 1 : most > 2048 ? 2048 : most;
    hipLaunchKernelGGL(chain_prepare, dim3((unsigned)grid), dim3(kNT), 0, st, static_cast<uint4 *>(q.workspace), count, q.cu,
                       q.B, q.T, q.D, from, to);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (ch.tiles == 0) return hipSuccess;
  ch.by_die = ch.chains * ch.tiles > kSpread ? ch.tiles / kDies * kDies * ch.chains : 0;
  const dim3 grid((unsigned)((size_t)ch.chains * ch.tiles));
  if (op == kForward) {
    if (q.cu) hipLaunchKernelGGL((linear_forward_chain<BF16, FORM, VEC, true>), grid, dim3(kNT), 0, st, p, ch);
    else hipLaunchKernelGGL((linear_forward_chain<BF16, FORM, VEC, false>), grid, dim3(kNT), 0, st, p, ch);
  } else {
    if (q.cu) hipLaunchKernelGGL((linear_backward_chain<BF16, FORM, VEC, true>), grid, dim3(kNT), 0, st, p, ch);
    else hipLaunchKernelGGL((linear_backward_chain<BF16, FORM, VEC, false>), grid, dim3(kNT), 0, st, p, ch);
  }
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

size_t linear_chain_bytes(int B, int T, int D, bool packed) {
  return chain_bytes((packed ? 1 : B) * ((D + kLinChannels - 1) / kLinChannels), (T + kLinTile - 1) / kLinTile);
}

hipError_t launch_linear_forward(const LinearArgs &q, hipStream_t st) { return launch(q, kForward, st); }

hipError_t launch_linear_backward(const LinearArgs &q, hipStream_t st) {
  LinearArgs p = q;
  if (!p.ck) {  // the saved states again: a forward pass that writes nothing else
    p.ck = reinterpret_cast<float *>(static_cast<char *>(p.workspace) + linear_chain_bytes(p.B, p.T, p.D, p.cu != nullptr));
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
