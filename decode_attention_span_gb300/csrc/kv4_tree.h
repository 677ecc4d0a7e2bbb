// Attention of many (token, head) columns over the 4-bit cache (kv4_tree.cu), for kv4_attn.cu.
#pragma once

#include "kv4.cuh"

namespace sekv {

constexpr int kTreeRows = 128;      // (token, head) columns of a group
constexpr int kTreeItems = 304;     // pieces of groups, where groups are cut: two for each SM
constexpr size_t kTreePartialFloats = size_t(kTreeRows) * (kHeadDim + 2);
// What a stream has flushed, in the order of its 128 threads: values, then sums and a reference of each of four rows
constexpr size_t kTreeKeptFloats = size_t(kTreeRows) * (kHeadDim + 16);
inline size_t tree_bytes(int sms) { return (kTreeItems * kTreePartialFloats + size_t(sms) * 2 * kTreeKeptFloats) * 4; }

// Groups (sequence, block of columns, KV head) as items of at most `piece` pages each.
struct TreePlan {
  int before[SEKV_KV4_MAX_BATCH + 1];  // items before each sequence
  int len[SEKV_KV4_MAX_BATCH];         // tokens of each sequence, drafted ones among them
  int piece;                           // pages
};

struct TreeCall {
  Kv4Pages pg;
  const void* q;
  const int32_t* first;
  const int64_t* tree;
  int64_t tree_stride;
  float *out, *lse, *partials;
  float* kept;  // [CTA][stream][kTreeKeptFloats]
  uint64_t wait_ns;
  int batch, hpg, n_q, n_blk, bf16;
  float scale_log2;
};
sekv_status tree_attention(const TreeCall& call, int sms, cudaStream_t stream);

}  // namespace sekv
