// gdn2_attention_api.cpp -- the C ABI of the attention layer: the head norm with
// its rotation by position, softmax attention, its decode step over a paged
// key-value cache and that cache's writes (include/gdn2.h): argument checks,
// then a launch on the caller's stream.
#include "gdn2.h"

#include <math.h>

#include <initializer_list>

#include "gdn2_attention.hpp"
#include "gdn2_check.hpp"
#include "gdn2_rotary.hpp"

using gdn2::aligned16;
using gdn2::aligned4;
using gdn2::aligned_to;
using gdn2::ceil_div;
using gdn2::kMaxGroups;
using gdn2::Range;
using gdn2::range_of;

namespace {

gdn2_status status_of(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP; }
bool known(int dtype) { return dtype == GDN2_F32 || dtype == GDN2_BF16; }
size_t size_of(int dtype) { return dtype == GDN2_BF16 ? 2 : 4; }

// Rows of `width` values, `stride` values apart (0: one behind the other).
int64_t stride_of(int64_t stride, int64_t width) { return stride ? stride : width; }
size_t strided(int64_t rows, int64_t stride, int64_t width, size_t es) {
  return rows > 0 ? ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * es : 0;
}

// ------------------------------------------------------------------ head norm and rotation
constexpr int64_t kMaxStride = 1 << 22;

gdn2_status check_rotary(const gdn2_rotary_desc *d) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (!known(d->dtype) || !known(d->wdtype)) return GDN2_ERR_BAD_DTYPE;
  if (d->tokens < 0 || d->H_q < 0 || d->H_k < 0 || d->d < 1 || d->rot < 0 || d->rot > d->d || !(d->eps >= 0.f) || isinf(d->eps))
    return GDN2_ERR_BAD_SHAPE;
  if (d->d % 2 || d->rot % 2 || d->d > gdn2::kRotaryMaxD || (d->pairs != GDN2_PAIRS_HALVES && d->pairs != GDN2_PAIRS_NEIGHBOURS))
    return GDN2_ERR_UNSUPPORTED;
  const int64_t wq = (int64_t)d->H_q * d->d, wk = (int64_t)d->H_k * d->d;
  if (wq > kMaxStride || wk > kMaxStride || d->stride_q > kMaxStride || d->stride_k > kMaxStride || d->tokens > INT32_MAX)
    return GDN2_ERR_UNSUPPORTED;
  if ((d->stride_q && d->stride_q < wq) || (d->stride_k && d->stride_k < wk)) return GDN2_ERR_BAD_SHAPE;
  return GDN2_OK;
}

gdn2::RotaryArgs rotary_args(const gdn2_rotary_desc *d, const void *q, const void *k, const void *qw, const void *kw,
                             const int32_t *positions, const float *inv_freq) {
  gdn2::RotaryArgs p{};
  p.tokens = d->tokens;
  p.Hq = d->H_q; p.Hk = d->H_k; p.d = d->d; p.rot = d->rot;
  p.norm = d->norm != 0;
  p.neighbours = d->pairs == GDN2_PAIRS_NEIGHBOURS;
  p.bf16 = d->dtype == GDN2_BF16;
  p.wbf16 = d->wdtype == GDN2_BF16;
  p.eps = d->eps;
  p.sq = stride_of(d->stride_q, (int64_t)d->H_q * d->d);
  p.sk = stride_of(d->stride_k, (int64_t)d->H_k * d->d);
  p.q = q; p.k = k; p.qw = qw; p.kw = kw;
  p.positions = positions;
  p.inv_freq = inv_freq;
  return p;
}

// ------------------------------------------------------------------ attention
gdn2_status check_attention(const gdn2_attention_desc *d, bool packed, bool backward) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (!known(d->dtype)) return GDN2_ERR_BAD_DTYPE;
  if (d->B < 0 || d->T_q < 0 || d->T_k < 0 || d->H < 1 || d->H_kv < 1 || d->H % d->H_kv || d->window < 0 || !(d->scale > 0.f) ||
      isinf(d->scale))
    return GDN2_ERR_BAD_SHAPE;
  if ((d->d != 64 && d->d != 128) || (d->window && !d->causal)) return GDN2_ERR_UNSUPPORTED;
  const int64_t wq = (int64_t)d->H * d->d, wk = (int64_t)d->H_kv * d->d;
  if (wq > kMaxStride || d->stride_q > kMaxStride || d->stride_k > kMaxStride || d->stride_v > kMaxStride) return GDN2_ERR_UNSUPPORTED;
  if ((d->stride_q && d->stride_q < wq) || (d->stride_k && d->stride_k < wk) || (d->stride_v && d->stride_v < wk))
    return GDN2_ERR_BAD_SHAPE;
  const size_t es = size_of(d->dtype);
  if (d->stride_q * es % 16 || d->stride_k * es % 16 || d->stride_v * es % 16) return GDN2_ERR_BAD_SHAPE;
  if (d->T_q > INT32_MAX - 256 || d->T_k > INT32_MAX - 256) return GDN2_ERR_UNSUPPORTED;
  // workgroups: blocks of 128 rows, and a head each; in the backward, 512 threads or twice as many blocks of 64 keys
  const size_t most = backward ? kMaxGroups / 2 : kMaxGroups, B = (size_t)d->B;
  for (const int T : {d->T_q, d->T_k}) {
    const size_t blocks = gdn2::attention_blocks(d->B, T, gdn2::kAttnRows, packed);
    if (blocks > most || B > most || blocks * (size_t)d->H > most || (!packed && blocks * (size_t)d->H * B > most))
      return GDN2_ERR_UNSUPPORTED;
  }
  return GDN2_OK;
}

int64_t q_rows(const gdn2_attention_desc *d, bool packed) { return (packed ? 1 : (int64_t)d->B) * d->T_q; }
int64_t k_rows(const gdn2_attention_desc *d, bool packed) { return (packed ? 1 : (int64_t)d->B) * d->T_k; }

gdn2::AttentionArgs attention_args(const gdn2_attention_desc *d) {
  gdn2::AttentionArgs p{};
  p.B = d->B; p.Tq = d->T_q; p.Tk = d->T_k; p.H = d->H; p.Hkv = d->H_kv; p.d = d->d;
  p.bf16 = d->dtype == GDN2_BF16;
  p.causal = d->causal != 0;
  p.window = d->window >= d->T_k ? 0 : d->window;  // as wide as the keys: every one of them
  p.scale = d->scale;
  p.sq = stride_of(d->stride_q, (int64_t)d->H * d->d);
  p.sk = stride_of(d->stride_k, (int64_t)d->H_kv * d->d);
  p.sv = stride_of(d->stride_v, (int64_t)d->H_kv * d->d);
  return p;
}

gdn2_status attention_forward(const gdn2_attention_desc *d, bool packed, const int32_t *cu_q, const int32_t *cu_k, const void *q,
                              const void *k, const void *v, void *o, float *lse, void *stream) {
  const gdn2_status st = check_attention(d, packed, false);
  if (st != GDN2_OK) return st;
  const int64_t nq = q_rows(d, packed), nk = k_rows(d, packed);
  if (d->B == 0 || nq == 0) return GDN2_OK;
  if (!q || !o || (nk && (!k || !v)) || (packed && (!cu_q || !cu_k))) return GDN2_ERR_NULL_POINTER;
  for (const void *x : {q, k, v, (const void *)o})
    if (!aligned16(x)) return GDN2_ERR_BAD_SHAPE;
  if (!aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_k)) return GDN2_ERR_BAD_SHAPE;
  gdn2::AttentionArgs p = attention_args(d);
  const size_t es = size_of(d->dtype), cu = packed ? ((size_t)d->B + 1) * 4 : 0;
  const int64_t w = (int64_t)d->H * d->d, wk = (int64_t)d->H_kv * d->d;
  const Range in[] = {range_of(q, strided(nq, p.sq, w, es)), range_of(k, strided(nk, p.sk, wk, es)),
                      range_of(v, strided(nk, p.sv, wk, es)), range_of(cu_q, cu), range_of(cu_k, cu)};
  const Range out[] = {range_of(o, (size_t)nq * w * es), range_of(lse, lse ? (size_t)nq * d->H * 4 : 0)};
  if (gdn2::outputs_overlap(in, 5, out, 2, nullptr)) return GDN2_ERR_ALIAS;
  p.cu_q = packed ? cu_q : nullptr;
  p.cu_k = packed ? cu_k : nullptr;
  p.q = q; p.k = k; p.v = v; p.o = o; p.lse = lse;
  return status_of(gdn2::launch_attention_forward(p, reinterpret_cast<hipStream_t>(stream)));
}

// delta, lse in powers of two, and the parts' sums of dk and dv, each from a multiple of 16 bytes on
struct BackwardSpace {
  size_t rows, partial, bytes;
  gdn2::AttentionSplit split;
};
BackwardSpace backward_space(const gdn2_attention_desc *d, bool packed) {
  BackwardSpace s;
  s.rows = ceil_div((size_t)q_rows(d, packed) * d->H * 4, 16) * 16;
  s.split = gdn2::attention_backward_split(d->B, d->T_k, d->H, d->H_kv, d->d, d->dtype == GDN2_BF16,
                                           attention_args(d).window, packed);
  s.partial = s.split.parts > 1 ? (size_t)s.split.parts * 2 * k_rows(d, packed) * d->H_kv * d->d * 4 : 0;
  s.bytes = 2 * s.rows + s.partial;
  return s;
}
size_t attention_backward_ws(const gdn2_attention_desc *d, bool packed) {
  return check_attention(d, packed, true) != GDN2_OK || d->B == 0 ? 0 : backward_space(d, packed).bytes;
}

gdn2_status attention_backward(const gdn2_attention_desc *d, bool packed, const int32_t *cu_q, const int32_t *cu_k, const void *q,
                               const void *k, const void *v, const void *o, const float *lse, const void *dO, void *dq, void *dk,
                               void *dv, void *workspace, size_t workspace_bytes, void *stream) {
  const gdn2_status st = check_attention(d, packed, true);
  if (st != GDN2_OK) return st;
  const int64_t nq = q_rows(d, packed), nk = k_rows(d, packed);
  if (nq == 0 && nk == 0) return GDN2_OK;
  const size_t ws = attention_backward_ws(d, packed);
  if (ws && (!workspace || workspace_bytes < ws)) return GDN2_ERR_WORKSPACE;
  if ((nq && (!q || !o || !lse || !dO || !dq)) || (nk && (!k || !v || !dk || !dv)) || (packed && (!cu_q || !cu_k)))
    return GDN2_ERR_NULL_POINTER;
  for (const void *x : {q, k, v, o, dO, (const void *)dq, (const void *)dk, (const void *)dv})
    if (!aligned16(x)) return GDN2_ERR_BAD_SHAPE;
  if (!aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_k) || (ws && !aligned16(workspace))) return GDN2_ERR_BAD_SHAPE;
  gdn2::AttentionArgs p = attention_args(d);
  const size_t es = size_of(d->dtype), cu = packed ? ((size_t)d->B + 1) * 4 : 0;
  const int64_t w = (int64_t)d->H * d->d, wk = (int64_t)d->H_kv * d->d;
  const size_t bq = (size_t)nq * w * es, bk = (size_t)nk * wk * es;
  const Range in[] = {range_of(q, strided(nq, p.sq, w, es)), range_of(k, strided(nk, p.sk, wk, es)),
                      range_of(v, strided(nk, p.sv, wk, es)), range_of(o, bq), range_of(lse, (size_t)nq * d->H * 4),
                      range_of(dO, bq), range_of(cu_q, cu), range_of(cu_k, cu)};
  const Range out[] = {range_of(dq, bq), range_of(dk, bk), range_of(dv, bk), range_of(workspace, ws)};
  if (gdn2::outputs_overlap(in, 8, out, 4, nullptr)) return GDN2_ERR_ALIAS;
  p.cu_q = packed ? cu_q : nullptr;
  p.cu_k = packed ? cu_k : nullptr;
  p.q = q; p.k = k; p.v = v; p.o_in = o; p.lse_in = lse; p.dO = dO;
  p.dq = dq; p.dk = dk; p.dv = dv;
  if (d->B > 0) {
    const BackwardSpace s = backward_space(d, packed);
    char *at = static_cast<char *>(workspace);
    p.delta = reinterpret_cast<float *>(at);
    p.lse = reinterpret_cast<float *>(at + s.rows);
    p.partial = reinterpret_cast<float *>(at + 2 * s.rows);
    p.keys = s.split.keys;
    p.parts = s.split.parts;
  }
  return status_of(gdn2::launch_attention_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ decode and cache
bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

gdn2_status check_decode(const gdn2_attention_decode_desc *d) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (!known(d->dtype)) return GDN2_ERR_BAD_DTYPE;
  if (d->N < 0 || d->P < 0 || d->M < 0 || d->H < 1 || d->H_kv < 1 || d->H % d->H_kv || d->window < 0 || d->page < 1 ||
      !(d->scale > 0.f) || isinf(d->scale))
    return GDN2_ERR_BAD_SHAPE;
  if ((d->d != 64 && d->d != 128) || !power_of_two(d->page) || (int64_t)d->M * d->page > 1 << 30) return GDN2_ERR_UNSUPPORTED;
  const gdn2::DecodePlan plan = gdn2::decode_plan(d->N, d->H, d->H_kv, d->M, d->page, d->window);
  const size_t heads = (size_t)d->N * d->H;
  // a join of 1024 threads a head
  if (heads > kMaxGroups / 4 || (size_t)d->N * d->H_kv * plan.tiles * plan.splits > kMaxGroups) return GDN2_ERR_UNSUPPORTED;
  return GDN2_OK;
}

size_t decode_ws(const gdn2_attention_decode_desc *d) {
  if (check_decode(d) != GDN2_OK || d->N == 0) return 0;
  return gdn2::decode_workspace_bytes(gdn2::decode_plan(d->N, d->H, d->H_kv, d->M, d->page, d->window), d->N, d->H, d->d);
}

gdn2_status check_store(const gdn2_kv_cache_desc *d, bool packed) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (!known(d->dtype)) return GDN2_ERR_BAD_DTYPE;
  const int64_t w = (int64_t)d->H_kv * d->d;
  if (d->N < 0 || d->T < 0 || d->P < 0 || d->M < 0 || d->H_kv < 1 || d->page < 1 || (!packed && d->T != d->N)) return GDN2_ERR_BAD_SHAPE;
  if ((d->d != 64 && d->d != 128) || !power_of_two(d->page) || (int64_t)d->M * d->page > 1 << 30 || w > kMaxStride ||
      d->stride_k > kMaxStride || d->stride_v > kMaxStride || d->T > INT32_MAX - 256 || d->N > INT32_MAX - 256)
    return GDN2_ERR_UNSUPPORTED;
  if ((d->stride_k && d->stride_k < w) || (d->stride_v && d->stride_v < w) || d->stride_k * size_of(d->dtype) % 16 ||
      d->stride_v * size_of(d->dtype) % 16)
    return GDN2_ERR_BAD_SHAPE;
  return GDN2_OK;
}

}  // namespace

extern "C" {

gdn2_status gdn2_rotary_forward(const gdn2_rotary_desc *d, const void *q, const void *k, const void *q_weight, const void *k_weight,
                                const int32_t *positions, const float *inv_freq, void *q_out, void *k_out, void *stream) {
  const gdn2_status st = check_rotary(d);
  if (st != GDN2_OK) return st;
  if (d->tokens == 0 || (d->H_q == 0 && d->H_k == 0)) return GDN2_OK;
  if ((d->H_q && (!q || !q_out)) || (d->H_k && (!k || !k_out)) || !positions || (d->rot && !inv_freq)) return GDN2_ERR_NULL_POINTER;
  const size_t es = size_of(d->dtype), ws = size_of(d->wdtype);
  for (const void *x : {q, k, (const void *)q_out, (const void *)k_out})
    if (!aligned_to(x, es)) return GDN2_ERR_BAD_SHAPE;
  if (!aligned_to(q_weight, ws) || !aligned_to(k_weight, ws) || !aligned4(positions) || !aligned4(inv_freq)) return GDN2_ERR_BAD_SHAPE;
  gdn2::RotaryArgs p = rotary_args(d, q, k, q_weight, k_weight, positions, inv_freq);
  const int64_t wq = (int64_t)d->H_q * d->d, wk = (int64_t)d->H_k * d->d;
  const Range in[] = {range_of(q, d->H_q ? strided(d->tokens, p.sq, wq, es) : 0),
                      range_of(k, d->H_k ? strided(d->tokens, p.sk, wk, es) : 0),
                      range_of(q_weight, q_weight ? d->d * ws : 0),
                      range_of(k_weight, k_weight ? d->d * ws : 0),
                      range_of(positions, (size_t)d->tokens * 4),
                      range_of(inv_freq, (size_t)d->rot * 2)};
  const Range out[] = {range_of(q_out, (size_t)d->tokens * wq * es), range_of(k_out, (size_t)d->tokens * wk * es)};
  if (gdn2::outputs_overlap(in, 6, out, 2, nullptr)) return GDN2_ERR_ALIAS;
  p.q_out = q_out;
  p.k_out = k_out;
  return status_of(gdn2::launch_rotary_forward(p, reinterpret_cast<hipStream_t>(stream)));
}

size_t gdn2_rotary_backward_workspace_bytes(const gdn2_rotary_desc *d) {
  return check_rotary(d) != GDN2_OK ? 0 : gdn2::rotary_backward_workspace_bytes(d->tokens, d->H_q, d->H_k, d->d);
}

gdn2_status gdn2_rotary_backward(const gdn2_rotary_desc *d, const void *q, const void *k, const void *q_weight, const void *k_weight,
                                 const int32_t *positions, const float *inv_freq, const void *gq, const void *gk, void *dq, void *dk,
                                 void *dq_weight, void *dk_weight, void *workspace, size_t workspace_bytes, void *stream) {
  const gdn2_status st = check_rotary(d);
  if (st != GDN2_OK) return st;
  const size_t need = dq_weight || dk_weight ? gdn2_rotary_backward_workspace_bytes(d) : 0;
  if (need && (!workspace || workspace_bytes < need)) return GDN2_ERR_WORKSPACE;
  const bool rows = d->tokens > 0 && (d->H_q || d->H_k);
  if (rows && ((d->H_q && (!q || !gq || !dq)) || (d->H_k && (!k || !gk || !dk)) || !positions || (d->rot && !inv_freq)))
    return GDN2_ERR_NULL_POINTER;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return GDN2_ERR_NULL_POINTER;
  const size_t es = size_of(d->dtype), ws = size_of(d->wdtype);
  for (const void *x : {q, k, gq, gk, (const void *)dq, (const void *)dk})
    if (!aligned_to(x, es)) return GDN2_ERR_BAD_SHAPE;
  for (const void *x : {q_weight, k_weight, (const void *)dq_weight, (const void *)dk_weight})
    if (!aligned_to(x, ws)) return GDN2_ERR_BAD_SHAPE;
  if (!aligned4(positions) || !aligned4(inv_freq) || (need && !aligned16(workspace))) return GDN2_ERR_BAD_SHAPE;
  gdn2::RotaryArgs p = rotary_args(d, q, k, q_weight, k_weight, positions, inv_freq);
  const int64_t wq = (int64_t)d->H_q * d->d, wk = (int64_t)d->H_k * d->d;
  const size_t nq = (size_t)d->tokens * wq * es, nk = (size_t)d->tokens * wk * es, nw = d->d * ws;
  const Range in[] = {range_of(q, d->H_q ? strided(d->tokens, p.sq, wq, es) : 0),
                      range_of(k, d->H_k ? strided(d->tokens, p.sk, wk, es) : 0),
                      range_of(q_weight, q_weight ? nw : 0),
                      range_of(k_weight, k_weight ? nw : 0),
                      range_of(positions, (size_t)d->tokens * 4),
                      range_of(inv_freq, (size_t)d->rot * 2),
                      range_of(gq, nq),
                      range_of(gk, nk)};
  const Range out[] = {range_of(dq, nq), range_of(dk, nk), range_of(dq_weight, dq_weight ? nw : 0),
                       range_of(dk_weight, dk_weight ? nw : 0), range_of(workspace, need)};
  if (gdn2::outputs_overlap(in, 8, out, 5, nullptr)) return GDN2_ERR_ALIAS;
  if (!rows) p.tokens = 0;
  p.gq = gq; p.gk = gk; p.dq = dq; p.dk = dk; p.dqw = dq_weight; p.dkw = dk_weight;
  p.workspace = workspace;
  return status_of(gdn2::launch_rotary_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_attention_forward(const gdn2_attention_desc *d, const void *q, const void *k, const void *v, void *o, float *lse,
                                   void *stream) {
  return attention_forward(d, false, nullptr, nullptr, q, k, v, o, lse, stream);
}

gdn2_status gdn2_attention_forward_varlen(const gdn2_attention_desc *d, const int32_t *cu_q, const int32_t *cu_k, const void *q,
                                          const void *k, const void *v, void *o, float *lse, void *stream) {
  return attention_forward(d, true, cu_q, cu_k, q, k, v, o, lse, stream);
}

size_t gdn2_attention_backward_workspace_bytes(const gdn2_attention_desc *d) { return attention_backward_ws(d, false); }
size_t gdn2_attention_backward_varlen_workspace_bytes(const gdn2_attention_desc *d) { return attention_backward_ws(d, true); }

gdn2_status gdn2_attention_backward(const gdn2_attention_desc *d, const void *q, const void *k, const void *v, const void *o,
                                    const float *lse, const void *dO, void *dq, void *dk, void *dv, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  return attention_backward(d, false, nullptr, nullptr, q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, stream);
}

gdn2_status gdn2_attention_backward_varlen(const gdn2_attention_desc *d, const int32_t *cu_q, const int32_t *cu_k, const void *q,
                                           const void *k, const void *v, const void *o, const float *lse, const void *dO, void *dq,
                                           void *dk, void *dv, void *workspace, size_t workspace_bytes, void *stream) {
  return attention_backward(d, true, cu_q, cu_k, q, k, v, o, lse, dO, dq, dk, dv, workspace, workspace_bytes, stream);
}

size_t gdn2_attention_decode_workspace_bytes(const gdn2_attention_decode_desc *d) { return decode_ws(d); }

gdn2_status gdn2_attention_decode(const gdn2_attention_decode_desc *d, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *pages, const int32_t *lengths, void *o, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  const gdn2_status st = check_decode(d);
  if (st != GDN2_OK) return st;
  if (d->N == 0) return GDN2_OK;
  const size_t ws = decode_ws(d);
  if (ws && (!workspace || workspace_bytes < ws)) return GDN2_ERR_WORKSPACE;
  if (!q || !lengths || !o || (d->P && (!k_cache || !v_cache)) || (d->M && !pages)) return GDN2_ERR_NULL_POINTER;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned4(pages) || !aligned4(lengths) ||
      (ws && !aligned16(workspace)))
    return GDN2_ERR_BAD_SHAPE;
  const size_t es = size_of(d->dtype), nq = (size_t)d->N * d->H * d->d * es, nc = (size_t)d->P * d->H_kv * d->page * d->d * es;
  const Range in[] = {range_of(q, nq), range_of(k_cache, nc), range_of(v_cache, nc), range_of(pages, (size_t)d->N * d->M * 4),
                      range_of(lengths, (size_t)d->N * 4)};
  const Range out[] = {range_of(o, nq), range_of(workspace, ws)};
  if (gdn2::outputs_overlap(in, 5, out, 2, nullptr)) return GDN2_ERR_ALIAS;
  gdn2::DecodeArgs p{};
  p.N = d->N; p.H = d->H; p.Hkv = d->H_kv; p.d = d->d; p.P = d->P; p.page = d->page; p.M = d->M;
  p.bf16 = d->dtype == GDN2_BF16;
  p.window = d->window;
  p.scale = d->scale;
  p.q = q; p.kc = k_cache; p.vc = v_cache; p.pages = pages; p.lengths = lengths; p.o = o;
  p.workspace = static_cast<float *>(workspace);
  return status_of(gdn2::launch_attention_decode(p, reinterpret_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_kv_cache_store(const gdn2_kv_cache_desc *d, const int32_t *cu_seqlens, const void *k, const void *v,
                                const int32_t *pages, const int32_t *lengths, void *k_cache, void *v_cache, void *stream) {
  const gdn2_status st = check_store(d, cu_seqlens != nullptr);
  if (st != GDN2_OK) return st;
  if (d->N == 0 || d->T == 0 || d->P == 0 || d->M == 0) return GDN2_OK;
  if (!k || !v || !pages || !lengths || !k_cache || !v_cache) return GDN2_ERR_NULL_POINTER;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned4(pages) || !aligned4(lengths) ||
      !aligned4(cu_seqlens))
    return GDN2_ERR_BAD_SHAPE;
  gdn2::StoreArgs p{};
  p.N = d->N; p.T = d->T; p.Hkv = d->H_kv; p.d = d->d; p.P = d->P; p.page = d->page; p.M = d->M;
  p.bf16 = d->dtype == GDN2_BF16;
  const int64_t w = (int64_t)d->H_kv * d->d;
  p.sk = stride_of(d->stride_k, w);
  p.sv = stride_of(d->stride_v, w);
  const size_t es = size_of(d->dtype), nc = (size_t)d->P * w * d->page * es;
  const Range in[] = {range_of(k, strided(d->T, p.sk, w, es)), range_of(v, strided(d->T, p.sv, w, es)),
                      range_of(pages, (size_t)d->N * d->M * 4), range_of(lengths, (size_t)d->N * 4),
                      range_of(cu_seqlens, cu_seqlens ? ((size_t)d->N + 1) * 4 : 0)};
  const Range out[] = {range_of(k_cache, nc), range_of(v_cache, nc)};
  if (gdn2::outputs_overlap(in, 5, out, 2, nullptr)) return GDN2_ERR_ALIAS;
  p.cu = cu_seqlens;
  p.k = k; p.v = v; p.pages = pages; p.lengths = lengths; p.kc = k_cache; p.vc = v_cache;
  return status_of(gdn2::launch_kv_cache_store(p, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
