/*
 * paged_attn_q8.h -- C ABI of a paged key/value cache held in 8 bits: the
 * operators that write it and read it back, and the attention over it.
 *
 * The pages are those of paged_attn_cache.h, 16 tokens each, with 8-bit codes
 * and one scale for each page and KV head:
 *
 *     k_cache  [num_blocks, num_kv_heads, head_size / 16, 16, 16]
 *     v_cache  [num_blocks, num_kv_heads, head_size, 16]
 *     k_scale, v_scale   float [num_blocks, num_kv_heads]
 *
 *     key[d]   = k_scale[page][g] * k_cache[page][g][d / 16][slot][d % 16]
 *     value[d] = v_scale[page][g] * v_cache[page][g][d][slot]
 *
 * where token p of sequence i stands in slot p % 16 of page
 * block_tables[i][p / 16].  A code is an e4m3 number (largest 448, 0x7f and
 * 0xff are NaN) or a two's complement integer (-127 .. 127 as written; -128 is
 * read as it is).  Scales are finite and >= 0; any other counts as NaN.
 *
 * Common to the calls: the rules of paged_attn_cache.h on pointers (caches,
 * keys, values, queries and outputs 16-byte aligned, arrays of int32 and float
 * 4-byte), streams, threads, block_size (16), head_size (64, 128 or 256) and
 * counts.  cu_seqlens int32 [num_seqs + 1] is taken as clipped to [0,
 * total_tokens]; a negative slice is empty; slices do not overlap.  Sequence i
 * has n_i = cu_seqlens[i + 1] - cu_seqlens[i] packed rows, which stand for the
 * last n_i of its seq_lens[i] tokens.  A page id outside [0, num_blocks) is
 * never used as an address: its tokens are skipped, and attn_varlen_check on
 * the same stream returns ATTN_VARLEN_ERR_BAD_BLOCK_TABLE.  num_seqs == 0 or
 * total_tokens == 0 returns ATTN_VARLEN_OK and launches nothing.
 *
 * Of the operators of paged_attn_cache.h, paged_attn_cache_free, which moves no
 * contents, works on these pages; write, accept, fork and compact take 16-bit
 * caches only.
 */
#ifndef PAGED_ATTN_Q8_H_
#define PAGED_ATTN_Q8_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime.h>

#include "attn_varlen.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of the codes. */
#define PAGED_ATTN_Q8_E4M3 0
#define PAGED_ATTN_Q8_INT8 1

/*
 * paged_attn_cache_write_q8 -- keys and values of new tokens are quantised into
 * the cache, in place.
 *
 * For each page that gets new tokens, KV head and each of keys and values: with
 * `largest` the largest finite magnitude among the new elements and
 *
 *     need = the smallest power of two, at least 2^-126, with
 *            largest <= 448 * need  (127 * need for integers),
 *
 * the page's scale becomes need, if the sequence has no tokens in the page
 * before the new ones; else the larger of need and its scale so far, rounded up
 * to a power of two (to 2^127, the largest there is, from above it).  New
 * elements x become the code nearest to x / scale, ties to even.  Where the
 * scale changed, the codes of the page's earlier tokens are rounded anew: the
 * code nearest to code * (old scale / new scale), the largest code where that is
 * past it (under an old scale above 2^127 only).  A scale that was raised stays
 * raised: a draft that is rejected and written over later leaves its page's
 * scale, and its earlier tokens' codes, as it made them.
 *
 * A non-finite element becomes NaN (e4m3), or -127, 0 or 127 for -infinity, NaN
 * and infinity (integers).  An old scale that is not finite and > 0 counts as
 * smaller than need; the earlier tokens' codes then are what the arithmetic
 * above makes of them.
 *
 *   key, value   device [total_tokens, num_kv_heads, head_size] of dtype
 *                (PAGED_ATTN_BF16 or PAGED_ATTN_FP16), strided as for
 *                paged_attn_cache_write
 *
 * A token whose position is negative is not written; nor is one at or past
 * max_blocks_per_seq * 16 (ATTN_VARLEN_ERR_BAD_BLOCK_TABLE).  Codes of slots
 * past a page's new tokens keep their bytes, as do other pages.  Pages that are
 * written are not shared between rows; k_cache and v_cache, and k_scale and
 * v_scale, share no memory (else ATTN_VARLEN_ERR_INVALID_ARG).
 */
int paged_attn_cache_write_q8(const void* key, const void* value, void* k_cache, void* v_cache,
                              float* k_scale, float* v_scale, const int32_t* block_tables,
                              const int32_t* seq_lens, const int32_t* cu_seqlens, int num_seqs,
                              int total_tokens, int num_kv_heads, int head_size, int block_size,
                              int max_blocks_per_seq, int num_blocks, int dtype, int code,
                              int64_t key_token_stride, int64_t key_head_stride,
                              int64_t value_token_stride, int64_t value_head_stride,
                              cudaStream_t stream);

/*
 * paged_attn_cache_read_q8 -- tokens are read back as 16-bit keys and values.
 *
 * Row cu_seqlens[i] + j receives token seq_lens[i] - n_i + j: scale * code in 32
 * bits, cut to the finite range of dtype, rounded once (NaN stays NaN).  So
 * seq_lens = b, n = b - a reads positions [a, b), and n = seq_lens all of them.
 *
 *   key, value   device [total_tokens, num_kv_heads, head_size] of dtype,
 *                strided as for paged_attn_cache_write, without rows or heads
 *                that share memory, in either or between the two; not
 *                overlapping the inputs.  Rows that no
 *                sequence covers, and those of negative positions, of positions
 *                at or past max_blocks_per_seq * 16 (ATTN_VARLEN_ERR_BAD_BLOCK_
 *                TABLE) and of bad pages, are not written
 */
int paged_attn_cache_read_q8(const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, const int32_t* block_tables,
                             const int32_t* seq_lens, const int32_t* cu_seqlens, int num_seqs,
                             int total_tokens, int num_kv_heads, int head_size, int block_size,
                             int max_blocks_per_seq, int num_blocks, int dtype, int code,
                             void* key, void* value, int64_t key_token_stride,
                             int64_t key_head_stride, int64_t value_token_stride,
                             int64_t value_head_stride, cudaStream_t stream);

/* Bytes of workspace paged_attn_q8 needs (0 for an unsupported head_size). */
size_t paged_attn_q8_workspace_size(int head_size);

/*
 * paged_attn_q8 -- attention of each sequence's last tokens over the cache.
 *
 * The keys and values of the n_i tokens are in the cache already.  Row
 * cu_seqlens[i] + j is token t = seq_lens[i] - n_i + j and sees the positions 0
 * .. t; query head h reads KV head g = h / (Hq / Hkv):
 *
 *     out[row, h, :] = sum over p <= t of w_p value_p,
 *     w = softmax over p <= t of scale * query[row, h, :] . key_p.
 *
 * For decoding (n_i = 1) and a few new or drafted tokens; longer runs are right
 * too, but their contexts are read again for every 8, 16, 24 or 32 rows (8 or 16
 * for head_size 256) of tokens x Hq / Hkv, by what the batch's sequences have on
 * average: a long run among many single tokens for every 8.  What a row does not
 * see (later tokens, unused slots, pages with a bad id, positions below 0 or
 * past the table) has no part in it, whatever it holds.  A row that sees nothing
 * gets zeros.  A query row with a non-finite element gives NaN if it sees
 * anything.
 *
 * Codes are exact operands of 16-bit products with sums in 32 bits.  A bf16
 * query row is taken as fp16 times a power of two, exact for elements above
 * 2^-31 of its largest and within 2^-39 of the largest otherwise.  Weights, with
 * the page's scale of the values, are rounded to fp16 for the value product
 * (products of weight and scale below 2^-32 of the row's largest may count as
 * 0), and the output once.  Queries, scale and key scales may be of any size in
 * their ranges, whether or not they make up for each other; scores that, times
 * log2 e, pass 2^100 are told apart to 2^-19 of themselves.
 *
 *   query, out    device [total_q, num_query_heads, head_size] of dtype, 16-byte
 *                 aligned, not overlapping (else ATTN_VARLEN_ERR_INVALID_ARG);
 *                 rows of out that no sequence covers are not written
 *   cu_seqlens    as above over total_q rows, or null: one row a sequence, in
 *                 order (total_q is num_seqs then)
 *   scale         > 0 and at most 2^126, or <= 0 for head_size^-1/2
 *   workspace     device buffer of paged_attn_q8_workspace_size(head_size)
 *                 bytes, 16-byte aligned, its contents free; calls that can
 *                 overlap on the GPU need one each
 */
int paged_attn_q8(const void* query, const void* k_cache, const void* v_cache,
                  const float* k_scale, const float* v_scale, const int32_t* block_tables,
                  const int32_t* seq_lens, const int32_t* cu_seqlens, int num_seqs, int total_q,
                  int num_query_heads, int num_kv_heads, int head_size, int block_size,
                  int max_blocks_per_seq, int num_blocks, float scale, int dtype, int code,
                  void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_ATTN_Q8_H_ */
