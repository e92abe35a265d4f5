/*
 * exl3_attn.h -- C ABI of what stands between a decoder's quantized q/k/v and
 * output projections on an MI355X (gfx950): rotary positions, a paged key and
 * value cache that is quantized as it is written, attention over that cache
 * and attention over packed prompts.  Same library (libexl3.so), status codes,
 * data types and error text (exl3_last_error) as exl3.h.
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers unless marked HOST.  The caller owns every
 *     buffer and the stream; no call allocates, frees or synchronizes, so all
 *     calls may be captured in a HIP graph.
 *   - Launches are made on the calling thread's current device, which has to
 *     be the buffers' and the stream's.
 *   - Every argument that is known on the host is checked before any HIP
 *     call; on error nothing is enqueued and exl3_last_error() names the
 *     failed check.  Values in device memory (positions, slots, lengths, page
 *     numbers) cannot be checked there: each call says what the kernels do
 *     with one that is out of range.  None makes them read or write outside
 *     the buffers.
 *   - head_dim is 64, 128 or 256.  Data pointers are 16-byte aligned; strides
 *     count elements and are multiples of 8.
 *   - Results do not change from run to run: no sum's order depends on
 *     timing.  A row's bits may depend on the call's other sequences, since
 *     they decide how many parts a row's keys are split into.
 */
#ifndef EXL3_ATTN_H
#define EXL3_ATTN_H

#include "exl3.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of 16-bit values [tokens][heads][head_dim] with any token and head
 * stride (the last dimension dense), e.g. the q, k or v columns of one fused
 * projection's output. */
typedef struct exl3_rows {
  void *data;
  int64_t token_stride;
  int64_t head_stride;
  int32_t heads;
} exl3_rows;

/* Rotary positions.  Pair i of the head's first `rot` dims turns by the angle
 * whose cosine and sine table[position][i] holds:
 *   a' = a*cos - b*sin,  b' = b*cos + a*sin
 * in fp32 (each product and sum rounded), then one rounding to the type.
 * Dims from `rot` on are copied.  A position outside 0..positions-1 gives NaN
 * in the rotated dims. */
typedef struct exl3_rotary {
  const float *table;  /* [positions][rot/2][2]: cosine, sine               */
  int32_t positions;
  int32_t rot;         /* multiple of 16, at most head_dim                   */
  int32_t interleaved; /* 0: a = x[i], b = x[i + rot/2];
                          1: a = x[2i], b = x[2i + 1]                        */
} exl3_rotary;

/* A paged cache of keys and values.  Token slot s is offset s % page_size of
 * page s / page_size.
 *   bits 16: k, v hold the values, [pages][heads][page_size][head_dim]
 *   bits 8:  e4m3 codes, one byte a value
 *   bits 4:  e2m1 codes, two values in a byte (the even index in the low half)
 * With 8 and 4 bits k_scale, v_scale [pages][heads][page_size][head_dim/32]
 * hold a byte s per block of 32 values: value = code * 2^(s - 127).  The
 * exponent is the smallest that holds the block's largest magnitude (up to
 * 448 for e4m3; up to 7 for e2m1, whose largest code 6 is the nearest to
 * everything up to 7), within limits that make every value exact in `dtype`;
 * codes are rounded to nearest, ties to even.  A block with a NaN or an
 * infinity has s = 255 and reads as NaN.
 * Page strides are in bytes; within a page everything is dense. */
typedef struct exl3_kv_cache {
  void *k, *v;
  uint8_t *k_scale, *v_scale; /* NULL when bits is 16 */
  int64_t k_page_bytes, v_page_bytes;
  int64_t k_scale_page_bytes, v_scale_page_bytes;
  int32_t pages;
  int32_t page_size; /* a power of two, 16..1024; pages * page_size < 2^31 */
  int32_t heads;
  int32_t head_dim;
  int32_t dtype; /* exl3_dtype of the values */
  int32_t bits;  /* 16, 8 or 4 */
} exl3_kv_cache;

/* q_out = rope(q), k_out = rope(k) in one launch; k and k_out may both be
 * NULL.  positions int32 [tokens].  An output is either exactly its input
 * (same pointer and strides: in place) or does not overlap an input. */
exl3_status exl3_rope(const exl3_rotary *r, const int32_t *positions, int32_t tokens, int32_t head_dim, int32_t dtype,
                      const exl3_rows *q, const exl3_rows *q_out, const exl3_rows *k, const exl3_rows *k_out,
                      void *stream);

/* Writes k and v rows to the cache slots[token] (int32).  A slot outside
 * 0..pages*page_size-1 is skipped (padding tokens: -1); a slot that several
 * tokens name holds no defined values afterwards. */
exl3_status exl3_cache_write(const exl3_kv_cache *c, const exl3_rows *k, const exl3_rows *v, const int32_t *slots,
                             int32_t tokens, void *stream);

/* exl3_rope and exl3_cache_write of the rotated k in one launch, with the
 * same bits as the two calls.  k_out may be NULL (the rotated keys are then
 * only in the cache). */
exl3_status exl3_rope_cache_write(const exl3_kv_cache *c, const exl3_rotary *r, const int32_t *positions,
                                  const int32_t *slots, int32_t tokens, const exl3_rows *q, const exl3_rows *q_out,
                                  const exl3_rows *k, const exl3_rows *k_out, const exl3_rows *v, void *stream);

/* Reads the keys and values of slots[i] back, i < n, as values of the cache's
 * dtype.  A slot out of range reads as zeros. */
exl3_status exl3_cache_read(const exl3_kv_cache *c, const int32_t *slots, int32_t n, const exl3_rows *k_out,
                            const exl3_rows *v_out, void *stream);

/* Attention of new tokens over the cache.  Sequence s has the query rows
 * cu_q[s] .. cu_q[s+1]-1 (int32 [batch+1], non-decreasing, from 0 to tokens)
 * and kv_len[s] keys (int32 [batch]), the new tokens' own among them: its i-th
 * query stands at position p = kv_len - q_len + i and sees the keys 0..p, or
 * p-window+1..p when window > 0 (at most 2^30).  Key j is at offset
 * j % page_size of page page_table[s][j / page_size] (int32, row stride
 * page_table_stride, width page_table_width); a page outside 0..pages-1, or
 * past the width, is a hole whose keys nobody sees.  A length in kv_len counts
 * as 0 to 2^31 - 2^21.  Query head h reads the cache's head
 * h / (q.heads / heads).  Rows that see no key are zero.  An offset in cu_q
 * counts as at least those before it and at most tokens; rows that then belong
 * to no sequence are not written.
 *   out = softmax(scale * q k^T) v, products in the cache's dtype with fp32
 * sums, the probabilities rounded to that type for the second product.  out is
 * either exactly q (same pointer and strides: in place) or does not overlap q;
 * it never overlaps the cache.
 *   One kernel, for few rows a sequence or for many, serves the whole call and
 * is chosen by the average number of new tokens: chunks of a prompt and single
 * tokens are faster in two calls than together (a chunk of 500 tokens over 20000
 * keys 243 us, 63 single tokens over up to 8000 keys 120, both in one call 480). */
exl3_status exl3_paged_attention(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out, const int32_t *cu_q,
                                 const int32_t *kv_len, const int32_t *page_table, int64_t page_table_stride,
                                 int32_t page_table_width, int32_t batch, int32_t tokens, float scale, int32_t window,
                                 void *workspace, size_t workspace_bytes, void *stream);

/* Attention within packed sequences: sequence s is the rows cu[s]..cu[s+1]-1
 * of q, k and v (int32 [batch+1], as cu_q above).  causal: row i sees 0..i of
 * its sequence, else all of it; window > 0 (causal only) the last `window` of
 * those.  out is exactly q or does not overlap it, as above, and never overlaps
 * k or v.  k and v have the same heads, q a multiple of them, and token strides
 * of at most 2^22 (the kernels address a tile of keys by 32-bit offsets). */
exl3_status exl3_prompt_attention(const exl3_rows *q, const exl3_rows *k, const exl3_rows *v, const exl3_rows *out,
                                  const int32_t *cu, int32_t batch, int32_t tokens, int32_t head_dim, int32_t dtype,
                                  int32_t causal, int32_t window, float scale, void *workspace, size_t workspace_bytes,
                                  void *stream);

/* Workspace of either attention call with these sizes (0: none; also 0 with
 * exl3_last_error() set when they are invalid).  It starts with
 * EXL3_WORKSPACE_COUNTER_BYTES of counters that must be zero before the first
 * call and that every call leaves zero, like the workspace of exl3_linear,
 * which may be the same. */
size_t exl3_attention_workspace_bytes(int32_t batch, int32_t tokens, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim);

#ifdef __cplusplus
}
#endif
#endif /* EXL3_ATTN_H */
