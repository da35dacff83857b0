/*
 * paged_attn_tree.h -- C ABI of attention for drafted tokens over a paged cache.
 *
 * A verification step of speculative decoding: sequence i has seq_lens[i]
 * cached tokens, the last n_i = cu_seqlens[i + 1] - cu_seqlens[i] of which are
 * drafts (their keys and values are in the cache already, as
 * paged_attn_cache_write leaves them).  The drafts form a tree: draft j hangs
 * on draft parents[cu_seqlens[i] + j] < j of the same sequence, or on the
 * context (-1).  With base_i = seq_lens[i] - n_i and A(j) = j and its
 * ancestors, draft j sees the positions
 *
 *     V(j) = { 0, ..., base_i - 1 }  and  { base_i + a : a in A(j) }
 *
 * and every query head h, reading KV head g = h / (Hq / Hkv), gets
 *
 *     out[cu_seqlens[i] + j, h, :] = sum over p in V(j) of w_p value_p,
 *     w = softmax over V(j) of scale * query[cu_seqlens[i] + j, h, :] . key_p.
 *
 * Without parents the drafts form a chain (draft j sees drafts 0 .. j): a few
 * new tokens of a prompt, or one token (n_i = 1, plain decoding).  The cache
 * layouts, types and head sizes are those of paged_attn_decode
 * (paged_attn_decode.h).  What a row does not see has no part in it, whatever
 * it holds (NaN and infinities in unused slots or other branches included;
 * non-finite values that rows do see cost time, up to six times as much).  A
 * row that sees nothing gets zeros.  Accumulation is fp32; weights are rounded
 * to the cache type for the value product (in fp16 those below 2^-32 of the
 * row's largest may count as 0), and the output once.
 */
#ifndef PAGED_ATTN_TREE_H_
#define PAGED_ATTN_TREE_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "attn_varlen.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Drafts a sequence can have in one call. */
#define PAGED_ATTN_MAX_DRAFTS 256

/* Bytes of workspace paged_attn_tree needs (0 for an unsupported head_size). */
size_t paged_attn_tree_workspace_size(int head_size);

/*
 *   query         device [total_q, num_query_heads, head_size], 16-byte aligned
 *   k_cache, v_cache, block_tables, seq_lens   as for paged_attn_decode
 *   cu_seqlens    int32 device [num_seqs + 1], taken as clipped to [0, total_q];
 *                 a negative slice is empty, slices do not overlap
 *   parents       int32 device [total_q], or null for chains
 *   num_seqs, total_q   >= 0, num_seqs at most 2^30 (either 0: returns
 *                 ATTN_VARLEN_OK, launches nothing)
 *   scale         > 0 and at most 2^126, or <= 0 for head_size^-1/2
 *   dtype         PAGED_ATTN_BF16 (0) or PAGED_ATTN_FP16 (1)
 *   out           like query, not overlapping the inputs (over query:
 *                 ATTN_VARLEN_ERR_INVALID_ARG); rows that no sequence covers
 *                 are not written
 *   workspace     device buffer of paged_attn_tree_workspace_size(head_size)
 *                 bytes, 16-byte aligned, its contents free; calls that can
 *                 overlap on the GPU need one each
 *
 * Found on the device and reported by attn_varlen_check on the same stream: a
 * page id outside [0, num_blocks) (its tokens count as unseen,
 * ATTN_VARLEN_ERR_BAD_BLOCK_TABLE); a parent outside [-1, j) (read as -1) and
 * more than PAGED_ATTN_MAX_DRAFTS drafts (zero rows), both
 * ATTN_VARLEN_ERR_BAD_DRAFT.  Tokens past max_blocks_per_seq * 16, and
 * positions below 0 (fewer tokens than drafts), do not exist.
 */
int paged_attn_tree(const void* query, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* seq_lens,
                    const int32_t* cu_seqlens, const int32_t* parents, int num_seqs, int total_q,
                    int num_query_heads, int num_kv_heads, int head_size, int block_size,
                    int max_blocks_per_seq, int num_blocks, float scale, int dtype, void* out,
                    void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_TREE_H_ */
