// gdn2_attention_backward.hip -- gradients of softmax attention.
//
//   p_ij = exp(s_ij - lse_i)     dv_j = sum_i p_ij dO_i     dp_ij = dO_i . v_j
//   delta_i = dO_i . o_i         ds_ij = p_ij (dp_ij - delta_i)
//   dq_i = scale sum_j ds_ij k_j              dk_j = scale sum_i ds_ij q_i
//
// Two passes, each of which computes the scores and dp again: one by blocks of
// queries (dq; it also leaves delta and lse, in powers of two, for the other),
// one by blocks of keys (dk, dv, over the query heads that share them). That is
// 14 d flops a pair instead of the 10 d of a single pass, whose dq would have to
// be summed by atomics in an order of their own: here results are the same bits
// at every run. Scores are kept so that the rows of the product to come are the
// registers: keys for dq, queries for dk and dv.
#include "gdn2_attention_device.hpp"

namespace gdn2 {
namespace {

using namespace attn;

// ---------------------------------------------------------------- dq
template <bool BF16, int D>
__global__ void __launch_bounds__(256, BF16 ? 2 : 1) attention_dq_kernel(const AttentionArgs p, unsigned total, unsigned tiles) {
  using L = Tile<BF16, D>;
  constexpr int KT = BF16 ? 64 : 32, SUB = KT / 32, ES = BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[2][2][KT * L::ROW];
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

  const int wrow = row0 + 32 * wave, mine = wrow + (lane & 31), row = min(mine, m.nq - 1);
  const int wlast = min(wrow + 31, m.nq - 1);
  const int64_t at = ((sp.q0 + row) * (int64_t)p.H + head) * D * ES;  // the row in o, dO and dq
  Frag<BF16> q[D / 16], g[D / 16];
  load_row<BF16, D>(q, static_cast<const char *>(p.q) + ((sp.q0 + row) * p.sq + (int64_t)head * D) * ES, h);
  load_row<BF16, D>(g, static_cast<const char *>(p.dO) + at, h);
  float delta = 0.f;
  {
    Frag<BF16> o[D / 16];
    load_row<BF16, D>(o, static_cast<const char *>(p.o_in) + at, h);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int j = 0; j < 8; ++j) delta = __builtin_fmaf((float)o[kk].v[j], (float)g[kk].v[j], delta);
    delta = other_half_sum(delta);
  }
  arrived(q);
  arrived(g);
  float lse = p.lse_in[sp.rows + row] * kLog2e;
  pin_regs(lse);
  const float c = p.scale * kLog2e;
  if (mine < m.nq && h == 0) {
    p.delta[sp.rows + mine] = delta;
    p.lse[sp.rows + mine] = lse;
  }
  const int hi = m.hi(row), lo = m.lo(row);
  const int blast = min(row0 + kAttnRows - 1, m.nq - 1);
  const int t_lo = m.lo(row0) / KT, t_hi = (m.hi(blast) + KT) / KT;
  const int w_lo = m.lo(min(wrow, m.nq - 1)), w_hi = wrow <= wlast ? m.hi(wlast) : -1;
  const int b_lo = m.lo(blast), b_hi = m.hi(row0);
  const int all_lo = m.lo(max(wlast, 0)), all_hi = m.hi(min(wrow, m.nq - 1));

  floatx16 acc[D / 32];
#pragma unroll
  for (int b = 0; b < D / 32; ++b) acc[b] = zero16();
  if (t_lo < t_hi) {
    Dma<BF16, D, KT> ks, vs;
    ks.init(p.sk * ES, tid);
    vs.init(p.sv * ES, tid);
    ks.load(sm.tile[t_lo & 1][0], kbase, t_lo * KT, m.nk, wave);
    vs.load(sm.tile[t_lo & 1][1], vbase, t_lo * KT, m.nk, wave);
    for (int t = t_lo; t < t_hi; ++t) {
      const int key0 = t * KT;
      landed();
      __syncthreads();
      if (t + 1 < t_hi) {
        ks.load(sm.tile[(t + 1) & 1][0], kbase, key0 + KT, m.nk, wave);
        vs.load(sm.tile[(t + 1) & 1][1], vbase, key0 + KT, m.nk, wave);
      }
      char *kt = sm.tile[t & 1][0];
      const char *vt = sm.tile[t & 1][1];
      const bool live = key0 <= w_hi && key0 + KT > w_lo;
      Frag<BF16> ds[SUB][2];
      if (live) {
        const bool masked = key0 < all_lo || key0 + KT - 1 > all_hi;
        const int from = lo - key0 - 4 * h, to = hi - key0 - 4 * h;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          floatx16 s = zero16(), dp = zero16();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) s = mma<BF16>(s, L::along(kt, 32 * u + (lane & 31), kk, h), q[kk]);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) dp = mma<BF16>(dp, L::along(vt, 32 * u + (lane & 31), kk, h), g[kk]);
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], c, -lse)) * (dp[i] - delta);
          if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (32 * u + row_of(i, 0) < from || 32 * u + row_of(i, 0) > to) s[i] = 0.f;
          }
          // bf16: one rounding of each ds
          ds[u][0] = operand<BF16>(s, 0);
          ds[u][1] = operand<BF16>(s, 1);
        }
      }
      const bool bad = (key0 < b_lo || key0 + KT - 1 > b_hi) && clean<BF16, D, KT>(kt, sm.notes, tid);
      if (live) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int b = 0; b < D / 32; ++b) acc[b] = mma<BF16>(acc[b], L::across(kt, 32 * u + 16 * e, 32 * b, lane), ds[u][e]);
      }
      if (bad) poison<BF16, D, KT>(acc, sm.notes, lo - key0, hi - key0, h);
    }
  }
  if (mine < m.nq) store_row<BF16, D>(static_cast<char *>(p.dq) + at, acc, p.scale, h);
}

// ---------------------------------------------------------------- dk, dv
template <bool BF16, int D>
__global__ void __launch_bounds__(256, 1) attention_dkv_kernel(const AttentionArgs p, unsigned total, unsigned tiles) {
  using L = Tile<BF16, D>;
  constexpr int QT = 32, ES = BF16 ? 2 : 4;
  __shared__ __attribute__((aligned(16))) struct {
    char tile[2][2][QT * L::ROW];
    float stat[2][2][64];  // lse in powers of two and delta of a tile's rows (64 lanes land, 32 are used)
    Odd<BF16, D, QT> notes[2];
  } sm;
  unsigned unit, tile;
  if (!find_work(total, tiles, &unit, &tile)) return;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int group = p.H / p.Hkv, share = group / p.parts;  // query heads of a key head, and of this workgroup
  int seq, row0;
  const int part = (int)(unit % (unsigned)p.parts);
  unsigned kvu = unit / (unsigned)p.parts;
  if (p.cu_q) {
    if (!find_block(p.cu_k, p.B, p.Tk, (int)tile, &seq, &row0)) return;
  } else {
    seq = (int)(kvu / (unsigned)p.Hkv);
    kvu %= (unsigned)p.Hkv;
    row0 = (int)tile * kAttnRows;
  }
  const int kv = (int)kvu, head0 = kv * group + part * share;
  const Span sp = span_of(p, seq, head0);
  const Mask m = sp.m;
  if (row0 >= m.nk) return;

  const int wrow = row0 + 32 * wave, mine = wrow + (lane & 31), row = min(mine, m.nk - 1);
  const int wlast = min(wrow + 31, m.nk - 1);
  Frag<BF16> k[D / 16], v[D / 16];
  load_row<BF16, D>(k, static_cast<const char *>(p.k) + ((sp.k0 + row) * p.sk + (int64_t)kv * D) * ES, h);
  load_row<BF16, D>(v, static_cast<const char *>(p.v) + ((sp.k0 + row) * p.sv + (int64_t)kv * D) * ES, h);
  arrived(k);
  arrived(v);
  const float c = p.scale * kLog2e;
  const int first = m.first(row), last = m.last(row);
  // query tiles that some key of the workgroup, and of the wave, is seen from;
  // queries that see every key of them
  const int blast = min(row0 + kAttnRows - 1, m.nk - 1);
  const int t_lo = m.first(row0) / QT, t_hi = (m.last(blast) + QT) / QT;
  const int w_lo = m.first(min(wrow, m.nk - 1)), w_hi = wrow <= wlast ? m.last(wlast) : -1;
  const int b_lo = m.first(blast), b_hi = m.last(row0);
  const int all_lo = m.first(max(wlast, 0)), all_hi = m.last(min(wrow, m.nk - 1));

  floatx16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int b = 0; b < D / 32; ++b) dk[b] = dv[b] = zero16();
  const int nt = t_hi - t_lo;
  if (nt > 0) {
    Dma<BF16, D, QT> qs, gs;
    qs.init(p.sq * ES, tid);
    gs.init((int64_t)p.H * D * ES, tid);
    // tile t of head head0 + hd into buffer `to`
    auto fetch = [&](int hd, int t, int to) {
      const int head = head0 + hd, r0 = t * QT;
      qs.load(sm.tile[to][0], static_cast<const char *>(p.q) + (sp.q0 * p.sq + (int64_t)head * D) * ES, r0, m.nq, wave);
      gs.load(sm.tile[to][1], static_cast<const char *>(p.dO) + (sp.q0 * (int64_t)p.H + head) * D * ES, r0, m.nq, wave);
      if (wave < 2) {
        const float *from = (wave ? p.delta : p.lse) + sp.rows + (int64_t)hd * p.Tq + r0;
        dma<4>(reinterpret_cast<const char *>(from), (uint32_t)min(m.nq - r0, QT) * 4, lane * 4, lds_address(sm.stat[to][wave]));
      }
    };
    fetch(0, t_lo, 0);
    int hd = 0, t = t_lo;
    for (int it = 0; it < nt * share; ++it) {
      const int q0 = t * QT, buf = it & 1;
      landed();
      __syncthreads();
      if (++t == t_hi) t = t_lo, ++hd;
      if (hd < share) fetch(hd, t, buf ^ 1);
      char *qt = sm.tile[buf][0], *gt = sm.tile[buf][1];
      const float *ls = sm.stat[buf][0], *dl = sm.stat[buf][1];
      const bool live = q0 <= w_hi && q0 + QT > w_lo;
      Frag<BF16> pr[2], ds[2];
      if (live) {
        const bool masked = q0 < all_lo || q0 + QT - 1 > all_hi;
        floatx16 s = zero16(), dp = zero16();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) s = mma<BF16>(s, L::along(qt, lane & 31, kk, h), k[kk]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) dp = mma<BF16>(dp, L::along(gt, lane & 31, kk, h), v[kk]);
        const int from = first - q0 - 4 * h, to = last - q0 - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const floatx4 l4 = *reinterpret_cast<const floatx4 *>(ls + row_of(i, h));
          const floatx4 d4 = *reinterpret_cast<const floatx4 *>(dl + row_of(i, h));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[i + e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i + e], c, -l4[e]));
            dp[i + e] = s[i + e] * (dp[i + e] - d4[e]);
          }
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (row_of(i, 0) < from || row_of(i, 0) > to) s[i] = dp[i] = 0.f;
        }
        // bf16: one rounding of each p and ds
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          pr[e] = operand<BF16>(s, e);
          ds[e] = operand<BF16>(dp, e);
        }
      }
      bool bad_q = false, bad_g = false;
      if (q0 < b_lo || q0 + QT - 1 > b_hi) {
        bad_q = clean<BF16, D, QT>(qt, sm.notes[0], tid);
        bad_g = clean<BF16, D, QT>(gt, sm.notes[1], tid);
      }
      if (live) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int b = 0; b < D / 32; ++b) {
            dv[b] = mma<BF16>(dv[b], L::across(gt, 16 * e, 32 * b, lane), pr[e]);
            dk[b] = mma<BF16>(dk[b], L::across(qt, 16 * e, 32 * b, lane), ds[e]);
          }
      }
      if (bad_q) poison<BF16, D, QT>(dk, sm.notes[0], first - q0, last - q0, h);
      if (bad_g) poison<BF16, D, QT>(dv, sm.notes[1], first - q0, last - q0, h);
    }
  }
  if (mine >= m.nk) return;
  if (p.parts == 1) {
    const int64_t at = ((sp.k0 + mine) * (int64_t)p.Hkv + kv) * D * ES;
    store_row<BF16, D>(static_cast<char *>(p.dk) + at, dk, p.scale, h);
    store_row<BF16, D>(static_cast<char *>(p.dv) + at, dv, 1.f, h);
  } else {
    const int64_t n = (int64_t)(p.cu_q ? 1 : p.B) * p.Tk * p.Hkv * D;
    char *to = reinterpret_cast<char *>(p.partial + 2 * part * n + ((sp.k0 + mine) * (int64_t)p.Hkv + kv) * D);
    store_row<false, D>(to, dk, p.scale, h);
    store_row<false, D>(to + n * 4, dv, 1.f, h);
  }
}

// Sums of the parts, in order; four values a thread. Rows of no sequence are left to the next kernel.
template <bool BF16> __global__ void __launch_bounds__(256) attention_join_kernel(const AttentionArgs p, int64_t n) {
  const int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x), w = (int64_t)p.Hkv * p.d;
  if (i >= n) return;
  if (p.cu_q) {
    const int64_t token = i / w;
    if (token < clamp_to(p.cu_k[0], p.Tk) || token >= clamp_to(p.cu_k[p.B], p.Tk)) return;
  }
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
  const size_t units = packed ? 1 : (size_t)p.B;
  const size_t tq = attention_tiles(packed ? p.B : 1, p.Tq, packed), nq = tq * units * (size_t)p.H;
  if (nq) {
    attention_dq_kernel<BF16, D><<<(unsigned)((nq + 7) / 8 * 8), 256, 0, stream>>>(p, (unsigned)nq, (unsigned)tq);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const size_t tk = attention_tiles(packed ? p.B : 1, p.Tk, packed), nk = tk * units * (size_t)p.Hkv * (size_t)p.parts;
  if (nk) {
    attention_dkv_kernel<BF16, D><<<(unsigned)((nk + 7) / 8 * 8), 256, 0, stream>>>(p, (unsigned)nk, (unsigned)tk);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (nk && p.parts > 1) {
    const int64_t n = (int64_t)units * p.Tk * p.Hkv * D;
    attention_join_kernel<BF16><<<(unsigned)((n / 4 + 255) / 256), 256, 0, stream>>>(p, n);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// A key block's workgroup walks the query heads that share it. Where there are
// few such blocks the heads are dealt out to several workgroups, whose sums are
// joined in order: 4 workgroups a CU even out blocks that are seen by many
// queries and by few.
int attention_backward_parts(int B, int Tk, int H, int Hkv, bool packed) {
  const size_t blocks = (packed ? (size_t)Tk / kAttnRows + 1 : attention_tiles(1, Tk, false) * (size_t)B) * (size_t)Hkv;
  const int group = H / Hkv;
  for (int parts = 1; parts < group; ++parts)
    if (group % parts == 0 && blocks * parts >= 1024) return parts;
  return group;
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
