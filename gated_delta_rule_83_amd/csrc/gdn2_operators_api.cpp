// gdn2_operators_api.cpp -- the C ABI of the gated linear recurrence, the
// norms and the 8-bit state cache (include/gdn2.h): argument checks, then a
// launch on the caller's stream.
#include "gdn2.h"

#include <math.h>

#include <initializer_list>

#include "gdn2_check.hpp"
#include "gdn2_linear.hpp"
#include "gdn2_norm.hpp"
#include "gdn2_state_cache.hpp"

using gdn2::aligned16;
using gdn2::aligned4;
using gdn2::aligned_to;
using gdn2::ceil_div;
using gdn2::kMaxGroups;
using gdn2::overlaps;
using gdn2::Range;
using gdn2::range_of;

namespace {

gdn2_status status_of(hipError_t e) { return e == hipSuccess ? GDN2_OK : GDN2_ERR_HIP; }

gdn2_status check_overlap(const Range *in, int ni, const Range *out, int no, const int *same) {
  return gdn2::outputs_overlap(in, ni, out, no, same) ? GDN2_ERR_ALIAS : GDN2_OK;
}

// ------------------------------------------------------------------ linear recurrence
gdn2_status check_linear(const gdn2_linear_desc *d, bool packed) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) return GDN2_ERR_BAD_DTYPE;
  if (d->B < 0 || d->T < 0 || d->D < 1) return GDN2_ERR_BAD_SHAPE;
  if (d->gates < GDN2_LINEAR_CHANNEL || d->gates > GDN2_LINEAR_TIED_PREACT) return GDN2_ERR_UNSUPPORTED;
  // a tile's 64 token rows are addressed with 32-bit offsets
  if (d->T > INT32_MAX - 256 || d->D > 1 << 22) return GDN2_ERR_UNSUPPORTED;
  // workgroups: a tile of a chain each, and of whole sequences each has its own
  // chains; the products are below 2^25 * 2^15 and 2^24 * 2^31
  const size_t tiles = ceil_div((size_t)d->T, gdn2::kLinTile), blocks = ceil_div((size_t)d->D, gdn2::kLinChannels);
  const size_t per = (tiles > 0 ? tiles : 1) * blocks, B = (size_t)d->B;
  if (per > kMaxGroups || (packed ? B : per * B) > kMaxGroups) return GDN2_ERR_UNSUPPORTED;
  return GDN2_OK;
}

gdn2::LinearArgs linear_args(const gdn2_linear_desc *d) {
  gdn2::LinearArgs p{};
  p.B = d->B;
  p.T = d->T;
  p.D = d->D;
  p.gates = d->gates;
  p.bf16 = d->dtype == GDN2_BF16;
  return p;
}

bool tied_gates(int g) { return g == GDN2_LINEAR_TIED || g == GDN2_LINEAR_TIED_PREACT; }
bool pre_gates(int g) { return g == GDN2_LINEAR_PREACT || g == GDN2_LINEAR_TIED_PREACT; }

size_t linear_forward_ws(const gdn2_linear_desc *d, bool packed) {
  if (check_linear(d, packed) != GDN2_OK) return 0;
  return d->B == 0 ? 0 : gdn2::linear_chain_bytes(d->B, d->T, d->D, packed);
}

size_t linear_backward_ws(const gdn2_linear_desc *d, bool packed) {
  if (check_linear(d, packed) != GDN2_OK) return 0;
  if (d->B == 0 && !packed) return 0;
  return gdn2::linear_chain_bytes(d->B, d->T, d->D, packed) +
         gdn2::linear_checkpoint_rows(d->B, d->T, packed) * (size_t)d->D * 4;
}

gdn2_status linear_forward(const gdn2_linear_desc *d, bool packed, const int32_t *cu, const void *x, const void *a,
                           const void *b, const float *h0, void *o, float *h_T, float *ck, void *workspace,
                           size_t workspace_bytes, void *stream) {
  const gdn2_status st = check_linear(d, packed);
  if (st != GDN2_OK) return st;
  if (d->B == 0) return GDN2_OK;
  if (packed && !cu) return GDN2_ERR_NULL_POINTER;
  if (tied_gates(d->gates)) b = nullptr;
  const size_t ws = linear_forward_ws(d, packed);
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN2_ERR_WORKSPACE;
  const bool tokens = d->T > 0;
  if (tokens && (!x || !a || (!tied_gates(d->gates) && !b))) return GDN2_ERR_NULL_POINTER;
  if (!o && !h_T && !ck) return GDN2_ERR_NULL_POINTER;
  const size_t n = (packed ? 1 : (size_t)d->B) * d->T * d->D, ns = (size_t)d->B * d->D * 4;
  const size_t es = d->dtype == GDN2_BF16 ? 2 : 4, gs = pre_gates(d->gates) ? es : 4;
  if (!aligned_to(x, es) || !aligned_to(a, gs) || !aligned_to(b, gs) || !aligned_to(o, es) || !aligned4(h0) ||
      !aligned4(h_T) || !aligned4(ck) || !aligned4(cu) || (ws && !aligned16(workspace)))
    return GDN2_ERR_BAD_SHAPE;
  const Range in[] = {range_of(x, n * es), range_of(a, n * gs), range_of(b, b ? n * gs : 0), range_of(h0, h0 ? ns : 0),
                      range_of(cu, packed ? ((size_t)d->B + 1) * 4 : 0)};
  const Range out[] = {range_of(o, o ? n * es : 0), range_of(h_T, h_T ? ns : 0),
                       range_of(ck, ck ? gdn2::linear_checkpoint_rows(d->B, d->T, packed) * d->D * 4 : 0),
                       range_of(workspace, ws)};
  const int same[] = {-1, 3, -1, -1};
  const gdn2_status so = check_overlap(in, 5, out, 4, same);
  if (so != GDN2_OK) return so;
  gdn2::LinearArgs p = linear_args(d);
  p.x = x; p.a = a; p.b = b; p.h0 = h0; p.o = o; p.h_T = h_T; p.ck = ck;
  p.cu = packed ? cu : nullptr;
  p.workspace = workspace;
  return status_of(gdn2::launch_linear_forward(p, reinterpret_cast<hipStream_t>(stream)));
}

gdn2_status linear_backward(const gdn2_linear_desc *d, bool packed, const int32_t *cu, const void *x, const void *a,
                            const void *b, const float *h0, const float *ck, const void *dO, const float *dh_T,
                            void *dx, void *da, void *db, float *dh0, void *workspace, size_t workspace_bytes,
                            void *stream) {
  const gdn2_status st = check_linear(d, packed);
  if (st != GDN2_OK) return st;
  if (d->B == 0 && (!packed || d->T == 0)) return GDN2_OK;  // packed tokens of no sequence: gradients of zero
  if (packed && !cu) return GDN2_ERR_NULL_POINTER;
  if (tied_gates(d->gates)) b = db = nullptr;
  const size_t ws = linear_backward_ws(d, packed);
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN2_ERR_WORKSPACE;
  if (d->T > 0 && (!x || !a || !dO || !dx || !da || (!tied_gates(d->gates) && (!b || !db))))
    return GDN2_ERR_NULL_POINTER;
  const size_t n = (packed ? 1 : (size_t)d->B) * d->T * d->D, ns = (size_t)d->B * d->D * 4;
  const size_t es = d->dtype == GDN2_BF16 ? 2 : 4, gs = pre_gates(d->gates) ? es : 4;
  for (const void *p : {x, dO, (const void *)dx})
    if (!aligned_to(p, es)) return GDN2_ERR_BAD_SHAPE;
  for (const void *p : {a, b, (const void *)da, (const void *)db})
    if (!aligned_to(p, gs)) return GDN2_ERR_BAD_SHAPE;
  if (!aligned4(h0) || !aligned4(ck) || !aligned4(dh_T) || !aligned4(dh0) || !aligned4(cu) ||
      (ws && !aligned16(workspace)))
    return GDN2_ERR_BAD_SHAPE;
  const size_t nck = gdn2::linear_checkpoint_rows(d->B, d->T, packed) * d->D * 4;
  const Range in[] = {range_of(x, n * es), range_of(a, n * gs), range_of(b, b ? n * gs : 0), range_of(h0, h0 ? ns : 0),
                      range_of(ck, ck ? nck : 0), range_of(dO, n * es), range_of(dh_T, dh_T ? ns : 0),
                      range_of(cu, packed ? ((size_t)d->B + 1) * 4 : 0)};
  const Range out[] = {range_of(dx, n * es), range_of(da, n * gs), range_of(db, db ? n * gs : 0),
                       range_of(dh0, dh0 ? ns : 0), range_of(workspace, ws)};
  const int same[] = {-1, -1, -1, 6, -1};
  const gdn2_status so = check_overlap(in, 8, out, 5, same);
  if (so != GDN2_OK) return so;
  gdn2::LinearArgs p = linear_args(d);
  p.x = x; p.a = a; p.b = b; p.h0 = h0; p.ck = const_cast<float *>(ck); p.dO = dO; p.dh_T = dh_T;
  p.dx = dx; p.da = da; p.db = db; p.dh0 = dh0;
  p.cu = packed ? cu : nullptr;
  p.workspace = workspace;
  return status_of(gdn2::launch_linear_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------------------ norms
gdn2_status check_norm(const gdn2_norm_desc *d) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if ((d->dtype != GDN2_F32 && d->dtype != GDN2_BF16) || (d->wdtype != GDN2_F32 && d->wdtype != GDN2_BF16))
    return GDN2_ERR_BAD_DTYPE;
  if (d->rows < 0 || d->D < 1 || !(d->eps >= 0.f) || isinf(d->eps)) return GDN2_ERR_BAD_SHAPE;
  if (d->kind != GDN2_NORM_LAYER && d->kind != GDN2_NORM_RMS) return GDN2_ERR_UNSUPPORTED;
  // the columns' sums are one launch of a workgroup of 1024 threads for 16 columns
  if (d->D > 1 << 25 || (uint64_t)d->rows > (uint64_t)INT64_MAX / 8 / (uint64_t)d->D)
    return GDN2_ERR_UNSUPPORTED;
  return GDN2_OK;
}

gdn2::NormArgs norm_args(const gdn2_norm_desc *d, const void *x, const void *weight, const void *bias,
                         const void *gate) {
  gdn2::NormArgs p{};
  p.rows = d->rows;
  p.D = d->D;
  p.layer = d->kind == GDN2_NORM_LAYER;
  p.bf16 = d->dtype == GDN2_BF16;
  p.wbf16 = d->wdtype == GDN2_BF16;
  p.eps = d->eps;
  p.x = x; p.weight = weight; p.bias = bias; p.gate = gate;
  return p;
}

// Every tensor aligned to its elements: `wide` of desc->dtype, `cols` of desc->wdtype.
bool norm_aligned(const gdn2_norm_desc *d, std::initializer_list<const void *> wide,
                  std::initializer_list<const void *> cols) {
  for (const void *p : wide)
    if (!aligned_to(p, d->dtype == GDN2_BF16 ? 2 : 4)) return false;
  for (const void *p : cols)
    if (!aligned_to(p, d->wdtype == GDN2_BF16 ? 2 : 4)) return false;
  return true;
}

// ------------------------------------------------------------------ state cache
gdn2_status check_cache(const gdn2_cache_desc *d) {
  if (!d) return GDN2_ERR_NULL_POINTER;
  if (d->N < 0 || d->P < 0 || d->rows < 1 || d->d_v < 1) return GDN2_ERR_BAD_SHAPE;
  if (d->format != GDN2_CACHE_E4M3 && d->format != GDN2_CACHE_INT8) return GDN2_ERR_UNSUPPORTED;
  if (d->d_v != 16 && d->d_v != 32 && d->d_v != 64 && d->d_v != 128) return GDN2_ERR_UNSUPPORTED;
  if (d->rows > INT32_MAX - 4096 || gdn2::state_cache_groups(d->rows, d->d_v) * (size_t)d->N > kMaxGroups)
    return GDN2_ERR_UNSUPPORTED;
  return GDN2_OK;
}

gdn2_status state_cache(const gdn2_cache_desc *d, const float *S, const int32_t *slots, const void *cache,
                        const void *scales, bool store, void *stream) {
  const gdn2_status st = check_cache(d);
  if (st != GDN2_OK) return st;
  if (d->N == 0) return GDN2_OK;
  if (!S || !slots || (d->P > 0 && (!cache || !scales))) return GDN2_ERR_NULL_POINTER;
  if (!aligned16(S) || !aligned16(cache) || !aligned4(slots)) return GDN2_ERR_BAD_SHAPE;
  const size_t one = (size_t)d->rows;
  const Range rS = range_of(S, (size_t)d->N * one * d->d_v * 4), rslots = range_of(slots, (size_t)d->N * 4);
  const Range rc = range_of(cache, (size_t)d->P * one * d->d_v), rs = range_of(scales, (size_t)d->P * one);
  const Range all[] = {rS, rslots, rc, rs};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (overlaps(all[i], all[j])) return GDN2_ERR_ALIAS;
  gdn2::StateCacheArgs p{};
  p.N = d->N; p.P = d->P; p.rows = d->rows; p.d_v = d->d_v; p.format = d->format;
  p.S = const_cast<float *>(S);
  p.slots = slots;
  p.cache = static_cast<uint8_t *>(const_cast<void *>(cache));
  p.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
  const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  return status_of(store ? gdn2::launch_state_cache_store(p, hs) : gdn2::launch_state_cache_load(p, hs));
}

}  // namespace

extern "C" {

size_t gdn2_linear_forward_workspace_bytes(const gdn2_linear_desc *d) { return linear_forward_ws(d, false); }
size_t gdn2_linear_forward_varlen_workspace_bytes(const gdn2_linear_desc *d) { return linear_forward_ws(d, true); }
size_t gdn2_linear_backward_workspace_bytes(const gdn2_linear_desc *d) { return linear_backward_ws(d, false); }
size_t gdn2_linear_backward_varlen_workspace_bytes(const gdn2_linear_desc *d) { return linear_backward_ws(d, true); }

gdn2_status gdn2_linear_forward(const gdn2_linear_desc *d, const void *x, const void *a, const void *b,
                                const float *h0, void *o, float *h_T, float *ck, void *workspace,
                                size_t workspace_bytes, void *stream) {
  return linear_forward(d, false, nullptr, x, a, b, h0, o, h_T, ck, workspace, workspace_bytes, stream);
}

gdn2_status gdn2_linear_forward_varlen(const gdn2_linear_desc *d, const int32_t *cu_seqlens, const void *x,
                                       const void *a, const void *b, const float *h0, void *o, float *h_T, float *ck,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  return linear_forward(d, true, cu_seqlens, x, a, b, h0, o, h_T, ck, workspace, workspace_bytes, stream);
}

gdn2_status gdn2_linear_step(const gdn2_linear_desc *d, const void *x, const void *a, const void *b, const float *h,
                             float *h_out, void *o, void *stream) {
  const gdn2_status st = check_linear(d, false);
  if (st != GDN2_OK) return st;
  if (d->T != 1) return GDN2_ERR_BAD_SHAPE;
  if (d->B == 0) return GDN2_OK;
  if (tied_gates(d->gates)) b = nullptr;
  if (!x || !a || (!tied_gates(d->gates) && !b) || !h || !h_out || !o) return GDN2_ERR_NULL_POINTER;
  const size_t n = (size_t)d->B * d->D, es = d->dtype == GDN2_BF16 ? 2 : 4, gs = pre_gates(d->gates) ? es : 4;
  if (!aligned_to(x, es) || !aligned_to(a, gs) || !aligned_to(b, gs) || !aligned_to(o, es) || !aligned4(h) ||
      !aligned4(h_out))
    return GDN2_ERR_BAD_SHAPE;
  const Range in[] = {range_of(x, n * es), range_of(a, n * gs), range_of(b, b ? n * gs : 0), range_of(h, n * 4)};
  const Range out[] = {range_of(h_out, n * 4), range_of(o, n * es)};
  const int same[] = {3, -1};
  const gdn2_status so = check_overlap(in, 4, out, 2, same);
  if (so != GDN2_OK) return so;
  gdn2::LinearArgs p = linear_args(d);
  p.x = x; p.a = a; p.b = b; p.h0 = h; p.h_T = h_out; p.o = o;
  return status_of(gdn2::launch_linear_step(p, reinterpret_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_linear_backward(const gdn2_linear_desc *d, const void *x, const void *a, const void *b,
                                 const float *h0, const float *ck, const void *dO, const float *dh_T, void *dx,
                                 void *da, void *db, float *dh0, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  return linear_backward(d, false, nullptr, x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0, workspace, workspace_bytes,
                         stream);
}

gdn2_status gdn2_linear_backward_varlen(const gdn2_linear_desc *d, const int32_t *cu_seqlens, const void *x,
                                        const void *a, const void *b, const float *h0, const float *ck,
                                        const void *dO, const float *dh_T, void *dx, void *da, void *db, float *dh0,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  return linear_backward(d, true, cu_seqlens, x, a, b, h0, ck, dO, dh_T, dx, da, db, dh0, workspace, workspace_bytes,
                         stream);
}

gdn2_status gdn2_norm_forward(const gdn2_norm_desc *d, const void *x, const void *weight, const void *bias,
                              const void *gate, void *y, void *stream) {
  const gdn2_status st = check_norm(d);
  if (st != GDN2_OK) return st;
  if (d->rows == 0) return GDN2_OK;
  if (!x || !y) return GDN2_ERR_NULL_POINTER;
  if (!norm_aligned(d, {x, gate, y}, {weight, bias})) return GDN2_ERR_BAD_SHAPE;
  const size_t n = (size_t)d->rows * d->D * (d->dtype == GDN2_BF16 ? 2 : 4);
  const size_t nw = (size_t)d->D * (d->wdtype == GDN2_BF16 ? 2 : 4);
  const Range in[] = {range_of(x, n), range_of(weight, weight ? nw : 0), range_of(bias, bias ? nw : 0),
                      range_of(gate, gate ? n : 0)};
  const Range out[] = {range_of(y, n)};
  const int same[] = {-1};
  const gdn2_status so = check_overlap(in, 4, out, 1, same);
  if (so != GDN2_OK) return so;
  gdn2::NormArgs p = norm_args(d, x, weight, bias, gate);
  p.y = y;
  return status_of(gdn2::launch_norm_forward(p, reinterpret_cast<hipStream_t>(stream)));
}

size_t gdn2_norm_backward_workspace_bytes(const gdn2_norm_desc *d) {
  if (check_norm(d) != GDN2_OK) return 0;
  return gdn2::norm_backward_workspace_bytes(d->rows, d->D, d->dtype == GDN2_BF16);
}

gdn2_status gdn2_norm_backward(const gdn2_norm_desc *d, const void *x, const void *weight, const void *bias,
                               const void *gate, const void *dy, void *dx, void *dweight, void *dbias, void *dgate,
                               void *workspace, size_t workspace_bytes, void *stream) {
  const gdn2_status st = check_norm(d);
  if (st != GDN2_OK) return st;
  const size_t ws = dweight || dbias ? gdn2_norm_backward_workspace_bytes(d) : 0;
  if (ws > 0 && (!workspace || workspace_bytes < ws)) return GDN2_ERR_WORKSPACE;
  if (d->rows > 0 && (!x || !dy || !dx)) return GDN2_ERR_NULL_POINTER;
  if ((dweight && !weight) || (dbias && !bias) || (dgate && !gate)) return GDN2_ERR_NULL_POINTER;
  if (!norm_aligned(d, {x, gate, dy, dx, dgate}, {weight, bias, dweight, dbias}) || (ws && !aligned16(workspace)))
    return GDN2_ERR_BAD_SHAPE;
  const size_t n = (size_t)d->rows * d->D * (d->dtype == GDN2_BF16 ? 2 : 4);
  const size_t nw = (size_t)d->D * (d->wdtype == GDN2_BF16 ? 2 : 4);
  const Range in[] = {range_of(x, n), range_of(weight, weight ? nw : 0), range_of(bias, bias ? nw : 0),
                      range_of(gate, gate ? n : 0), range_of(dy, n)};
  const Range out[] = {range_of(dx, n), range_of(dweight, dweight ? nw : 0), range_of(dbias, dbias ? nw : 0),
                       range_of(dgate, dgate ? n : 0), range_of(workspace, ws)};
  const int same[] = {-1, -1, -1, -1, -1};
  const gdn2_status so = check_overlap(in, 5, out, 5, same);
  if (so != GDN2_OK) return so;
  gdn2::NormArgs p = norm_args(d, x, weight, bias, gate);
  p.dy = dy; p.dx = dx; p.dweight = dweight; p.dbias = dbias; p.dgate = dgate;
  p.workspace = workspace;
  return status_of(gdn2::launch_norm_backward(p, reinterpret_cast<hipStream_t>(stream)));
}

gdn2_status gdn2_state_cache_store(const gdn2_cache_desc *d, const float *S, const int32_t *slots, void *cache,
                                   void *scales, void *stream) {
  return state_cache(d, S, slots, cache, scales, true, stream);
}

gdn2_status gdn2_state_cache_load(const gdn2_cache_desc *d, const void *cache, const void *scales,
                                  const int32_t *slots, float *S, void *stream) {
  return state_cache(d, S, slots, cache, scales, false, stream);
}

}  // extern "C"
