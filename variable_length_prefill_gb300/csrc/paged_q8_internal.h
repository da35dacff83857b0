// Launch parameters of the 8-bit paged cache's operators (paged_q8_cache.cu,
// paged_q8_attn.cu), filled by the C ABI in attn_varlen_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "paged_cache_internal.h"

namespace avp {

// Tokens between the cache and packed rows, either way.
struct Q8MoveParams {
  CacheShape c;  // codes
  float* k_scale;
  float* v_scale;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu;
  int total_tokens;
  void* key;     // read by the write, written by the read
  void* value;
  long long key_token, key_head, value_token, value_head;  // strides, elements
};

struct Q8AttnParams {
  CacheShape c;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* cu;  // null: one row a sequence
  const void* query;
  void* out;
  uint8_t* workspace;
  int total_q;
  int num_query_heads;
  int group;         // query heads of a KV head
  float scale_log2;  // scale * log2(e)
  float scale_frac;  // the same as scale_frac * 2^scale_exp, scale_frac in [0.5, 1)
  int scale_exp;
  bool fp16;         // query and out, else bf16
  int test_withhold; // read only by test builds (ATTN_VARLEN_TEST_HOOKS); 0 otherwise
};

// The attention kernel's shape: query rows (new tokens x query heads of one KV head)
// of a tile, SMs it uses at most, one CTA on each, computing warps of a CTA.
constexpr int kQ8MaxRows = 32;
constexpr int kQ8MaxSms = 160;
constexpr int kQ8Warps = 8;
__host__ __device__ constexpr int q8_max_rows(int head_size) { return head_size == 256 ? 16 : kQ8MaxRows; }

// Workspace: a Q8Open record for each CTA, then fp32 partial results, two for each
// warp: four numbers for each row (the maximum, the exponent of O, the sum, one to
// spare), then O [rows][head_size].
struct Q8Open {
  int valid;       // a row tile that this CTA begins and leaves to others to finish
  int lo;          // first packed row of its sequence
  int n;           // rows of its sequence
  int g;           // KV head
  int tile;        // row tile
  int last;        // the CTA that holds its end
  int tail_piece;  // its piece here (in the CTAs behind it piece 0)
  int spare;
};

__host__ __device__ constexpr size_t q8_parts_offset() { return sizeof(Q8Open) * kQ8MaxSms; }
// floats of a piece: enough for the rows of any form
__host__ __device__ constexpr size_t q8_part_floats(int head_size, int rows) {
  return (size_t)rows * (head_size + 4);
}
__host__ __device__ constexpr size_t q8_form_bytes(int head_size, int rows) {
  return (size_t)2 * kQ8MaxSms * kQ8Warps * q8_part_floats(head_size, rows) *
         sizeof(float);
}
__host__ __device__ constexpr size_t q8_workspace_bytes(int head_size) {
  size_t most = 0;
  for (int rows = 8; rows <= q8_max_rows(head_size); rows *= 2) {
    const size_t bytes = q8_form_bytes(head_size, rows);
    if (bytes > most) most = bytes;
  }
  return q8_parts_offset() + most;
}

cudaError_t launch_q8_write(const Q8MoveParams& p, bool fp16, bool int8, cudaStream_t stream);
cudaError_t launch_q8_read(const Q8MoveParams& p, bool fp16, bool int8, cudaStream_t stream);
cudaError_t launch_q8_attn(const Q8AttnParams& p, bool int8, cudaStream_t stream);

}  // namespace avp
