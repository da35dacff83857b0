// Launch parameters of the tree attention kernels (paged_tree.cu), filled by
// the C ABI in attn_varlen_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "attn_varlen_internal.h"
#include "paged_cache_internal.h"

namespace avp {

constexpr int kTreeMaxDrafts = 256;

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
};

size_t tree_workspace_bytes(int head_size);
cudaError_t launch_tree(const TreeParams& p, bool fp16, EncodeTiledFn enc, cudaStream_t stream);

}  // namespace avp
