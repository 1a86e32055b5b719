/*
 * mxq_kv.h -- C ABI of libmxq, a paged MXFP8 key-value cache on GB300: quantizing keys and values as
 * they are written, reading them back as bf16, and the attention of one new token per sequence over
 * the cache, whose output may leave as the MXFP8 operand that o_proj_mxfp8 reads.
 *
 * The conventions, status codes, MXFP8 format and scale layouts are those of mxq.h: device pointers
 * owned by the caller, work enqueued on `stream`, argument errors detected on the host before anything
 * is launched, nothing allocated and nothing synchronized. Strides are below 2^40 bytes; that of a
 * dimension of size 1 is not looked at.
 *
 * No page describes these operators; they put the producer of o in front of the chain of mxq.h.
 */
#ifndef MXQ_KV_H_
#define MXQ_KV_H_

#include "mxq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache: `pages` pages of `page_size` tokens, each with `heads` rows of `dim` E4M3 values and
 * dim / 32 UE8M0 scale bytes (one per 32 consecutive values). The row of head h of the token at place r
 * of page p starts at data + p * page_stride + r * token_stride + h * head_stride, its scales at
 * sf + p * sf_page_stride + r * sf_token_stride + h * sf_head_stride (all in bytes), so both orders of
 * tokens and heads within a page can be had, and pages with other data between them. Rows of data start
 * on 16-byte boundaries; rows of scales on 4-byte boundaries where dim % 128 == 0, at strides below 2^31. Rows
 * must not overlap (strides, taken from the smallest up, each at least the span of those below it).
 * Slot s is place s % page_size of page s / page_size.
 * dim % 32 == 0, 32 <= dim <= 1024, heads <= 1024, page_size <= 65536, pages * page_size < 2^31.
 */
typedef struct mxq_kv_cache {
  void* data;
  void* sf;
  int64_t pages;
  int32_t page_size;
  int32_t heads;
  int32_t dim;
  int64_t page_stride, token_stride, head_stride;
  int64_t sf_page_stride, sf_token_stride, sf_head_stride;
} mxq_kv_cache;

/*
 * kv_write_mxfp8 -- quantizes rows as they are written into a cache:
 *   (k_cache row, scales)[slot[t], h] = mxfp8_quantize(k[t, h])     bit-identical; v likewise
 * A token whose slot lies outside [0, pages * page_size) is not written (-1: the padding of a batch).
 * The slots of one call must differ from one another.
 *
 *   k_bf16  [T, heads, dim] bf16, row strides ldk (tokens) and ldkh (heads) in elements.
 *   slots   [T] int32.
 *   v_bf16, v_cache : the values and their cache, or NULL, NULL. v_cache has k_cache's pages and page_size;
 *           its heads and dim may be others.
 * Requires T >= 1.
 */
MXQ_API mxq_status kv_write_mxfp8(const void* k_bf16, int64_t ldk, int64_t ldkh, const mxq_kv_cache* k_cache,
                                  const void* v_bf16, int64_t ldv, int64_t ldvh, const mxq_kv_cache* v_cache,
                                  const void* slots_i32, int64_t T, void* stream);

/*
 * kv_read_bf16 -- reads rows of sequences back:
 *   out[cu[b] + i, h] = RNE_bf16( deq(cache)[page table[b, p / page_size], place p % page_size, h] ),
 *   p = starts[b] + i, for 0 <= i < cu[b + 1] - cu[b]
 * (exact wherever the value is a normal bf16). Rows of a position outside the table, or of a page outside
 * [0, pages), are zero; rows outside [cu[0], cu[B]) are left as they were.
 *
 *   block_table [B, table_width] int32, row stride ld_table.
 *   cu_rows [B + 1] int32, not falling; starts [B] int32, or NULL for zeros.
 *   k_out   [rows, heads, dim] bf16, contiguous; v_cache, v_out: the values likewise, or NULL, NULL.
 * Requires B >= 1, rows >= 1, table_width >= 1.
 */
MXQ_API mxq_status kv_read_bf16(const mxq_kv_cache* k_cache, const mxq_kv_cache* v_cache, const void* block_table_i32,
                                int64_t ld_table, int32_t table_width, const void* cu_rows_i32, const void* starts_i32,
                                int64_t B, int64_t rows, void* k_out, void* v_out, void* stream);

/*
 * paged_attention_mxfp8 -- attention of one new token per sequence over the cache:
 *   s[b, h, t] = scale * sum_d q[b, h, d] * deq(k)[t, d]      over the sequence's tokens t < len_b, key head h / G
 *   o[b, h]    = RNE_bf16( sum_t softmax_t(s) * deq(v)[t] ),  lse[b, h] = ln sum_t exp(s)
 *   (o_q, scales) = mxfp8_quantize(o)                         of that bf16 o as [B, q_heads * dim], bit-identical
 * with G = q_heads / heads query heads for each head of the cache. Without a value cache the values are the
 * keys (a latent cache). Products and sums are in fp32. q enters them as the sum of two MXFP8 numbers (off by at
 * most 2^-21 of its group's largest magnitude), the probabilities in 16 bits (fp16, off by at most 2^-11 of itself or 2^-32 of the
 * largest so far; bf16 where the scales of a tile of values span more than fp16 holds). Values keep their precision beside scales up
 * to 2^100 times their own; further below the largest of their sequence and cache head they may lose bits or count as zeros, and so may
 * those of scale byte 0 (at most 448 * 2^-127) beside scales of 2^-112 and more.
 *
 * len_b = min(seq_lens[b], table_width * page_size); tokens on a page outside [0, pages) take no part. A
 * sequence without a token gives zeros and lse -inf. What the cache holds behind a sequence's end is not used,
 * NaN included. NaN among a sequence's tokens reaches its own outputs only; that of a value's scale (byte 255) all
 * features of its cache head's.
 *
 *   q_bf16   [B, q_heads, dim] bf16, row strides ldq (sequences) and ldqh (heads) in elements.
 *   v_cache  of k_cache's shape (strides may differ), or NULL.
 *   block_table [B, table_width] int32, row stride ld_table; seq_lens [B] int32.
 *   o_bf16   [B, q_heads, dim] bf16 out, or NULL.
 *   o_q      [B, q_heads * dim] E4M3 out and at least one scale output, or all NULL.
 *   lse_f32  [B, q_heads] fp32 out, or NULL.
 *   workspace: required, mxq_paged_attention_workspace_bytes(...) bytes, 16-byte aligned. Its contents need no
 *            clearing; calls that overlap in time need separate workspaces.
 *   status: optional device status word (mxq_status_bytes()).
 * At least one of o_bf16 and o_q. Requires dim in {128, 256, 384, 512}, page_size % 16 == 0, q_heads a multiple
 * of heads, q_heads <= 4096, 1 <= B <= 65536 / heads, table_width >= 1, table_width * page_size <= 2^30,
 * |scale| <= 1e38, and fewer than 2^30 pieces of 64 tokens: B * heads * ceil(q_heads / heads / 64) * ceil(table_width *
 * page_size / 64). o_bf16 may be q_bf16. Three launches; the results do not depend on timing.
 */
MXQ_API int64_t mxq_paged_attention_workspace_bytes(int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim);

MXQ_API mxq_status paged_attention_mxfp8(const void* q_bf16, int64_t ldq, int64_t ldqh, const mxq_kv_cache* k_cache,
                                         const mxq_kv_cache* v_cache, const void* block_table_i32, int64_t ld_table,
                                         int32_t table_width, const void* seq_lens_i32, int64_t B, int32_t q_heads,
                                         float scale, void* o_bf16, void* o_q, void* o_sf_packed_i32,
                                         void* o_sf_rowmajor, void* o_sf_128x4, void* lse_f32, void* workspace,
                                         int64_t workspace_bytes, void* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_KV_H_ */
