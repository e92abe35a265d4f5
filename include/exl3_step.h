/*
 * exl3_step.h -- C ABI of a serving step's operators beside those of
 * exl3_attn.h: block tables and slot maps from request lengths, the rotation
 * with norms of each query and key head and with several position axes,
 * attention with first tokens that stay visible beside a window, and
 * attention of sequences that share a prefix.  Same library, conventions
 * (streams, workspaces, checks before any HIP call, values in device memory
 * that are out of range), status codes and error text as exl3_attn.h.
 */
#ifndef EXL3_STEP_H
#define EXL3_STEP_H

#include "exl3_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rotary positions of several axes (time, height and width of a video's
 * patches): pair i turns by the angle that the table has for the token's
 * position on axis (axis_of[i / 16] >> 2 * (i % 16)) & 3, which is below axes.
 * positions are int32 [axes][tokens], rows axis_stride apart; one outside
 * 0..rotary.positions-1 gives NaN in the pairs of its axis. */
typedef struct exl3_rotary_axes {
  exl3_rotary rotary;
  int32_t axes;        /* 1..4 */
  uint32_t axis_of[8]; /* two bits a pair */
} exl3_rotary_axes;

/* Norms of each query and key head, before the rotation:
 *   n = x / sqrt(mean(x^2) + eps) * w
 * over the head's values.  w fp32: head_dim weights for all heads, or one such
 * row for each (q_rows, k_rows: 1 or the number of heads).  x * w stays within
 * fp32's range (it is taken before the division). */
typedef struct exl3_head_norm {
  const float *q, *k;
  int32_t q_rows, k_rows;
  float eps; /* 1e-30 .. 1 */
} exl3_head_norm;

/* exl3_rope with norms (n may be NULL: none) and axes: norm, rotation and one
 * rounding to the type, everything before it in fp32. */
exl3_status exl3_norm_rope(const exl3_rotary_axes *r, const exl3_head_norm *n, const int32_t *positions,
                           int64_t axis_stride, int32_t tokens, int32_t head_dim, int32_t dtype, const exl3_rows *q,
                           const exl3_rows *q_out, const exl3_rows *k, const exl3_rows *k_out, void *stream);

/* exl3_rope_cache_write with norms and axes; the same bits as exl3_norm_rope
 * and exl3_cache_write of its k_out. */
exl3_status exl3_norm_rope_cache_write(const exl3_kv_cache *c, const exl3_rotary_axes *r, const exl3_head_norm *n,
                                       const int32_t *positions, int64_t axis_stride, const int32_t *slots,
                                       int32_t tokens, const exl3_rows *q, const exl3_rows *q_out, const exl3_rows *k,
                                       const exl3_rows *k_out, const exl3_rows *v, void *stream);

/* What a step needs of its requests' lengths, in one launch.  Request b has
 * kv_len[b] tokens in a cache of `pages` pages of page_size tokens, on the pages
 * page_table[b][0..], and wants q_len[b] more.  The step has room for `tokens`
 * rows, which the requests get in order:
 *   cu_q [batch+1]   request b's rows are cu_q[b] .. cu_q[b+1]-1 (a request that
 *                    finds less room than it wants gets what is left)
 *   kv_out [batch]   kv_len and the new rows
 *   positions, slots [tokens]   of each row; rows that no request has: 0 and -1
 *   page_table       entries ceil(kv_len/page_size) .. ceil(kv_out/page_size)-1
 *                    (below width) become free_pages[taken], [taken+1], ... in the
 *                    order of the requests, -1 past n_free; other entries stay
 *   counts [2]       the rows that the requests wanted in all (at most 2^31-1), and the
 *                    entries that the table needed
 * taken: NULL (0) or one int32, the free pages used by earlier steps.  A row
 * whose page is not one of the cache's has slot -1.  q_len counts as 0..2^20,
 * kv_len as 0..2^30, taken as 0..n_free.  Outputs overlap neither inputs nor
 * each other; page_table (from its first row to the end of its last) is both. */
exl3_status exl3_cache_extend(int32_t pages, int32_t page_size, const int32_t *q_len, const int32_t *kv_len,
                              int32_t batch, int32_t *page_table, int64_t page_table_stride, int32_t page_table_width,
                              const int32_t *free_pages, int32_t n_free, const int32_t *taken, int32_t tokens,
                              int32_t *cu_q, int32_t *kv_out, int32_t *positions, int32_t *slots, int32_t *counts,
                              void *stream);

/* exl3_paged_attention and exl3_prompt_attention (causal) with a window of at
 * least 1 and first tokens that stay visible: a row at position p sees the keys
 * p-window+1..p and 0..sinks-1 (up to p), each once.  sinks is at most 2^20.
 * Pages that hold neither may be holes at no cost.  Workspace:
 * exl3_attention_workspace_bytes. */
exl3_status exl3_paged_attention_sinks(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out,
                                       const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                                       int64_t page_table_stride, int32_t page_table_width, int32_t batch,
                                       int32_t tokens, float scale, int32_t window, int32_t sinks, void *workspace,
                                       size_t workspace_bytes, void *stream);
exl3_status exl3_prompt_attention_sinks(const exl3_rows *q, const exl3_rows *k, const exl3_rows *v,
                                        const exl3_rows *out, const int32_t *cu, int32_t batch, int32_t tokens,
                                        int32_t head_dim, int32_t dtype, int32_t window, int32_t sinks, float scale,
                                        void *workspace, size_t workspace_bytes, void *stream);

/* exl3_paged_attention (without a window) of sequences that share prefixes.
 * Group g is the sequences group_cu[g] .. group_cu[g+1]-1 (int32 [groups+1],
 * non-decreasing, from 0 to batch; at most as many groups as sequences;
 * sequences of no group share nothing), whose rows of the page table, but for
 * sequences without new tokens, have the same pages for their first prefix_len[g]
 * (int32 [groups]) keys.  Of those, the keys before every new token of the
 * group's sequences are read once for all of them; the result is
 * exl3_paged_attention's but for the order of sums.  Calls that gain nothing by
 * it, by their sizes (few sequences, a narrow page table or more than 512 rows of a
 * sequence on each key/value head, on average), and those that would leave more
 * than 1 GiB between the passes are one launch of that, others two, or four of
 * 256 sequences and more.  The sizes are those that the host has: a page table
 * counts as full to its width.  One as wide as the longest sequence lets short
 * calls be one launch (4 sequences of 1100 keys, 8 heads of 128: 11 us; with a
 * table for 16384 keys or more they take the two passes, 18).  An offset in group_cu
 * counts as at least those before it and at most batch. */
exl3_status exl3_prefix_attention(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out,
                                  const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                                  int64_t page_table_stride, int32_t page_table_width, int32_t batch, int32_t tokens,
                                  const int32_t *group_cu, const int32_t *prefix_len, int32_t groups, float scale,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of exl3_prefix_attention, with counters at its start like that of
 * the other attention calls, which may be the same.  It does not depend on the
 * page table, so that what is reserved before a capture serves every table; it is
 * at most 1 GiB more than exl3_attention_workspace_bytes's and some arrays. */
size_t exl3_prefix_attention_workspace_bytes(int32_t batch, int32_t tokens, int32_t groups, int32_t q_heads,
                                             int32_t kv_heads, int32_t head_dim);

#ifdef __cplusplus
}
#endif
#endif /* EXL3_STEP_H */
