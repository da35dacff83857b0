// Launch parameters of the tree attention kernels (paged_tree.cu), filled by
// the C ABI in attn_varlen_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "paged_cache_internal.h"

namespace avp {

constexpr int kTreeMaxDrafts = 256;
constexpr int kTreeRows = 128;   // query rows of a tile (drafts x query heads of one KV head)
constexpr int kTreeMaxCtas = 160;  // CTAs of the attention kernel at most (one per SM)

struct TreeParams {
  CacheShape c;  // caches, status, sizes
  const void* query;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu;
  const int32_t* parents;  // null: chains
  void* out;
  uint8_t* workspace;
  int total_q;
  int num_query_heads;
  float scale_log2;  // scale * log2(e)
  int test_withhold; // read only by test builds (ATTN_VARLEN_TEST_HOOKS); 0 otherwise
};

// Workspace: kTreeMaxCtas TreeOpen records, then fp32 partial results
// [2 kTreeMaxCtas][head_size + 2][kTreeRows]: O, then the maximum (of scores
// without the scale) and the sum.
struct TreeOpen {
  int valid;  // a row tile that this CTA works on and leaves to others to finish
  int lo;     // first packed row of its sequence
  int n;      // drafts
  int g;      // KV head
  int mt;     // row tile
  int last;   // the CTA that finishes it
  int first;  // the CTA that began it
  int pad;
};

__host__ __device__ constexpr size_t tree_parts_offset() { return sizeof(TreeOpen) * kTreeMaxCtas; }
__host__ __device__ constexpr size_t tree_part_floats(int head_size) { return (size_t)(head_size + 2) * kTreeRows; }
__host__ __device__ constexpr size_t tree_workspace_bytes(int head_size) {
  return tree_parts_offset() + 2 * kTreeMaxCtas * tree_part_floats(head_size) * sizeof(float);
}

cudaError_t launch_tree(const TreeParams& p, bool fp16, cudaStream_t stream);

}  // namespace avp
