// Launch parameters of the paged-cache operators (paged_cache.cu), filled by
// the C ABI in attn_varlen_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace avp {

// Bits of the paged operators' device status word (a word of its own, apart
// from the attention workspaces' words, at a fixed address per device).
constexpr int kPageStatusBadBlock = 1;   // a page id, or a position past the table
constexpr int kPageStatusBadDraft = 2;   // a parent, an accepted index, too many drafts
constexpr int kPageStatusBadRow = 4;     // a row index, a page freed once too often
constexpr int kPageStatusNoBlock = 8;    // a fork found no free page
constexpr int kPageStatusTimeout = 16;   // a kernel wait ran out of time

constexpr int kPageTokens = 16;

// What every operator knows of the cache.
struct CacheShape {
  void* k_cache;   // [num_blocks, num_kv_heads, head_size / 8, 16, 8]
  void* v_cache;   // [num_blocks, num_kv_heads, head_size, 16]
  int* status;
  int num_seqs;
  int num_kv_heads;
  int head_size;
  int max_blocks;  // entries of a table row
  int num_blocks;
  int sm_count;
};

struct CacheWriteParams {
  CacheShape c;
  const void* key;
  const void* value;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu;
  int total_tokens;
  long long key_token, key_head, value_token, value_head;  // strides, elements
};

struct CacheAcceptParams {
  CacheShape c;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu;
  const int32_t* accepted;
  const int32_t* num_accepted;
  int max_accepted;
  int32_t* new_lens;
};

struct CacheFreeParams {
  CacheShape c;  // caches unused
  const int32_t* block_tables;
  int32_t* seq_lens;
  int32_t* refs;
  const int32_t* rows;
  int num_rows;
};

// Workspace of a fork: owner[num_seqs], is_src[num_seqs], state[num_forks],
// pages[num_forks], all int32.
struct CacheForkParams {
  CacheShape c;
  int32_t* block_tables;
  int32_t* seq_lens;
  int32_t* refs;
  const int32_t* src;
  const int32_t* dst;
  int num_forks;
  int32_t* owner;
  int32_t* is_src;
  int32_t* state;
  int32_t* pages;
};

// Workspace of a compaction, all int32: head (moves, used pages), then for every
// page the number of its move, and the moves' sources and targets.
struct CacheCompactParams {
  CacheShape c;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* refs;
  int32_t* block_tables_out;
  int32_t* refs_out;
  int32_t* head;
  int32_t* number;
  int32_t* from;
  int32_t* to;
};

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t stream);
cudaError_t launch_cache_accept(const CacheAcceptParams& p, cudaStream_t stream);
cudaError_t launch_cache_free(const CacheFreeParams& p, cudaStream_t stream);
cudaError_t launch_cache_fork(const CacheForkParams& p, cudaStream_t stream);
cudaError_t launch_cache_compact(const CacheCompactParams& p, cudaStream_t stream);

}  // namespace avp
