// gdn2_attention.hpp -- launch interface of softmax attention, its decode step
// over a paged key-value cache and that cache's writes (gdn2_attention_api.cpp
// to gdn2_attention*.hip). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

constexpr int kAttnRows = 128;   // queries of a workgroup (forward, dq)

struct AttentionArgs {
  int B, Tq, Tk, H, Hkv, d;   // packed: B sequences, Tq and Tk tokens in all
  bool bf16, causal;
  int window;                 // 0: none
  float scale;
  int64_t sq, sk, sv;         // elements from a token to the next
  const int32_t *cu_q, *cu_k; // null: B sequences of Tq and Tk tokens
  const void *q, *k, *v;
  void *o;
  float *lse;
  // backward
  const void *o_in, *dO;
  const float *lse_in;
  void *dq, *dk, *dv;
  float *delta;               // [lse] rowsum(dO o), from the dq pass to the dk, dv pass
  float *partial;             // parts > 1: [parts][2][rows of dk][Hkv * d]
  int keys, parts;            // AttentionSplit
};

// Blocks of `rows` queries (or keys) of one head: of one sequence, or (packed) of
// all B, each with room for a ragged last one.
inline size_t attention_blocks(int B, int T, int rows, bool packed) {
  return packed ? (size_t)T / rows + (size_t)B : ((size_t)T + rows - 1) / rows;
}
// The dk, dv pass: keys of a workgroup (64 or 128), and the workgroups that share
// a key block's query heads.
struct AttentionSplit {
  int keys, parts;
};
AttentionSplit attention_backward_split(int B, int Tk, int H, int Hkv, int d, bool bf16, int window, bool packed);

hipError_t launch_attention_forward(const AttentionArgs &p, hipStream_t stream);
hipError_t launch_attention_backward(const AttentionArgs &p, hipStream_t stream);

struct DecodeArgs {
  int N, H, Hkv, d, P, page, M; // M: columns of the page table
  bool bf16;
  int window;
  float scale;
  const void *q, *kc, *vc;
  const int32_t *pages, *lengths;
  void *o;
  float *workspace;
};

// Keys that one workgroup takes, and workgroups along the longest sequence.
struct DecodePlan {
  int span, splits, tiles;  // tiles: groups of 16 query heads that share a key head
};
DecodePlan decode_plan(int N, int H, int Hkv, int M, int page, int window);
size_t decode_workspace_bytes(const DecodePlan &plan, int N, int H, int d);
hipError_t launch_attention_decode(const DecodeArgs &p, hipStream_t stream);

struct StoreArgs {
  int N, T, Hkv, d, P, page, M;
  bool bf16;
  int64_t sk, sv;
  const int32_t *cu;  // null: one token a sequence
  const void *k, *v;
  const int32_t *pages, *lengths;
  void *kc, *vc;
};
hipError_t launch_kv_cache_store(const StoreArgs &p, hipStream_t stream);

}  // namespace gdn2
