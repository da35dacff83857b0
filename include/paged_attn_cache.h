/*
 * paged_attn_cache.h -- C ABI of the operators that fill and manage the paged
 * key/value cache that paged_attn_decode and paged_attn_tree read.
 *
 * Common to all of them.  The cache of one layer is
 *
 *     k_cache [num_blocks, num_kv_heads, head_size / 8, 16, 8]
 *     v_cache [num_blocks, num_kv_heads, head_size, 16]
 *
 * of 2-byte elements (bf16 or fp16; the calls below only move them).  Row i of
 * block_tables [num_seqs, max_blocks_per_seq] holds the pages of sequence i,
 * and seq_lens[i] its tokens: token p stands in slot p % 16 of page
 * block_tables[i][p / 16].  All pointers are caller-owned device pointers,
 * 16-byte aligned for caches, keys and values and 4-byte aligned for int32
 * arrays.  Calls are asynchronous on `stream`, read nothing back and allocate
 * nothing.  The index arrays live on the device, so what is wrong in them is
 * found there: the entry is skipped as described, and attn_varlen_check on the
 * same stream reports it.  Such a report stays until a check reads it.  Calls
 * may come from several threads; those on one stream act one after the other.
 *
 * A page id outside [0, num_blocks) is never used as an address
 * (ATTN_VARLEN_ERR_BAD_BLOCK_TABLE).  block_size is 16 and head_size 64, 128
 * or 256, as for paged_attn_decode.  num_seqs and the number of forks are at
 * most 2^30 (else ATTN_VARLEN_ERR_INVALID_ARG).  num_seqs == 0 (or no token,
 * row or fork to work on) returns ATTN_VARLEN_OK and launches nothing.
 */
#ifndef PAGED_ATTN_CACHE_H_
#define PAGED_ATTN_CACHE_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "attn_varlen.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * paged_attn_cache_write -- keys and values of new tokens go into the cache.
 *
 * Sequence i has n_i = cu_seqlens[i + 1] - cu_seqlens[i] new tokens (a
 * negative difference is none), packed rows cu_seqlens[i] on; seq_lens[i]
 * counts them already.  New token j gets position seq_lens[i] - n_i + j:
 *
 *     k_cache[page][g][d / 8][slot][d % 8] = key[row][g][d]
 *     v_cache[page][g][d][slot]            = value[row][g][d]
 *
 *   key, value   device [total_tokens, num_kv_heads, head_size]; the strides
 *                between tokens and between heads are given in elements, are
 *                >= 0 and multiples of 8; the head's elements are contiguous
 *   total_tokens packed rows; cu_seqlens is taken as clipped to
 *                [0, total_tokens], rows that no sequence covers are not used
 *
 * A token whose position is negative is not written; nor is one at or past
 * max_blocks_per_seq * 16 (ATTN_VARLEN_ERR_BAD_BLOCK_TABLE).  Every other slot
 * of the caches keeps its bytes.  Slots written by one call must be distinct:
 * pages that are written are not shared between rows.
 */
int paged_attn_cache_write(const void* key, const void* value, void* k_cache, void* v_cache,
                           const int32_t* block_tables, const int32_t* seq_lens,
                           const int32_t* cu_seqlens, int num_seqs, int total_tokens,
                           int num_kv_heads, int head_size, int block_size,
                           int max_blocks_per_seq, int num_blocks, int64_t key_token_stride,
                           int64_t key_head_stride, int64_t value_token_stride,
                           int64_t value_head_stride, cudaStream_t stream);

/*
 * paged_attn_cache_accept -- the accepted drafts move up to the context's end.
 *
 * The last n_i = cu_seqlens[i + 1] - cu_seqlens[i] tokens of sequence i are
 * drafts, from position base_i = seq_lens[i] - n_i on.  For m <
 * num_accepted[i], the keys and values of draft accepted[i][m] move to
 * position base_i + m, as if all were read before any is written, and
 *
 *     new_lens[i] = base_i + num_accepted[i]     (at least 0).
 *
 *   accepted      int32 [num_seqs, max_accepted], increasing within a row and
 *                 below n_i (the path from the context down a tree is)
 *   num_accepted  int32 [num_seqs], 0 .. max_accepted
 *   new_lens      int32 [num_seqs], not overlapping the inputs
 *
 * A row's acceptance ends before its first entry that is out of order or out
 * of range, and num_accepted is cut to [0, min(max_accepted, n_i)]; both are
 * ATTN_VARLEN_ERR_BAD_DRAFT.  A draft whose source or target page id is bad,
 * or whose position is negative, is not moved.  Written pages are not shared.
 */
int paged_attn_cache_accept(void* k_cache, void* v_cache, const int32_t* block_tables,
                            const int32_t* seq_lens, const int32_t* cu_seqlens,
                            const int32_t* accepted, const int32_t* num_accepted, int num_seqs,
                            int max_accepted, int num_kv_heads, int head_size, int block_size,
                            int max_blocks_per_seq, int num_blocks, int32_t* new_lens,
                            cudaStream_t stream);

/*
 * Page counts.  refs int32 [num_blocks] says how many rows hold each page; a
 * page with a count of 0 is free.  Whoever hands out pages by other means (a
 * server's allocator, for a prompt's pages) sets their counts to 1.
 */

/*
 * paged_attn_cache_free -- rows give their pages back.
 *
 * For each r = rows[j]: the counts of the pages of its ceil(seq_lens[r] / 16)
 * table entries go down by one and seq_lens[r] becomes 0; the table keeps its
 * bytes.  A row named twice is freed once.  A row outside [0, num_seqs), or a
 * page whose count is 0 already, is skipped (ATTN_VARLEN_ERR_BAD_ROW).
 */
int paged_attn_cache_free(const int32_t* block_tables, int32_t* seq_lens, int32_t* refs,
                          const int32_t* rows, int num_rows, int num_seqs, int block_size,
                          int max_blocks_per_seq, int num_blocks, cudaStream_t stream);

/* Bytes of workspace paged_attn_cache_fork needs (0 for a negative count). */
size_t paged_attn_cache_fork_workspace_size(int num_forks, int num_seqs);

/*
 * paged_attn_cache_fork -- rows become copies of others.
 *
 * For each j, row dst[j] becomes a copy of row src[j] as it stands before the
 * call: whole pages are shared (their counts go up by one); a last page that
 * holds fewer than 16 tokens is copied, keys and values, into a free page,
 * whose count becomes 1; seq_lens[dst[j]] = seq_lens[src[j]].  An id that is no
 * page is copied as it is.  Table entries past the pages keep their bytes.
 * Free pages are taken from the lowest id on, in order of j, so the result is
 * always the same.
 *
 * dst[j] has to be an empty row (seq_lens 0: freed, or never used), no src of
 * this call, and named once: of several j with the same dst the first counts.
 * The others, and those with src or dst outside [0, num_seqs), are refused
 * (ATTN_VARLEN_ERR_BAD_ROW); one that finds no free page is refused too
 * (ATTN_VARLEN_ERR_NO_FREE_BLOCK).  A refused fork changes nothing.
 *
 *   workspace  device buffer of paged_attn_cache_fork_workspace_size bytes,
 *              4-byte aligned, its contents free; calls that can overlap on
 *              the GPU need one each
 */
int paged_attn_cache_fork(void* k_cache, void* v_cache, int32_t* block_tables, int32_t* seq_lens,
                          int32_t* refs, const int32_t* src, const int32_t* dst, int num_forks,
                          int num_seqs, int num_kv_heads, int head_size, int block_size,
                          int max_blocks_per_seq, int num_blocks, void* workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* Bytes of workspace paged_attn_cache_compact needs (0 for a negative count). */
size_t paged_attn_cache_compact_workspace_size(int num_blocks);

/*
 * paged_attn_cache_compact -- the used pages move to the lowest ids.
 *
 * With U pages in use, the lowest free page below U receives the keys, values
 * and count of the highest used page, the next lowest those of the next
 * highest, until pages [0, U) are used and the others free.  The table's
 * entries for the ceil(seq_lens / 16) pages of each row follow; other entries
 * are copied as they are.
 *
 *   block_tables_out, refs_out  shaped like the inputs; each may be the input
 *                               itself (in place), else they do not overlap it
 *   workspace                   paged_attn_cache_compact_workspace_size bytes,
 *                               as for paged_attn_cache_fork
 */
int paged_attn_cache_compact(void* k_cache, void* v_cache, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* refs, int num_seqs,
                             int num_kv_heads, int head_size, int block_size,
                             int max_blocks_per_seq, int num_blocks, int32_t* block_tables_out,
                             int32_t* refs_out, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_CACHE_H_ */
