// Host side of the C ABI declared in include/exl3_attn.h: argument checks,
// the choice of kernel, and launches.  Every check runs before any HIP call.
#include "attn_checks.hpp"

namespace {

using namespace exl3;

// Either kernel of attn_small.hpp and attn_tile.hpp.
exl3_status run_plain(AttnParams &p, int32_t head_dim, bool bf16, int32_t bits, int32_t q_heads, void *workspace,
                      size_t workspace_bytes, hipStream_t s) {
  return run_attention(p, head_dim, q_heads, workspace, workspace_bytes, [&](int columns) {
    return columns > 0 ? launch_attn_small(head_dim, bf16, bits, p, columns, s) : launch_attn_tile(head_dim, bf16, bits, p, s);
  });
}

}  // namespace

namespace exl3 {

hipError_t launch_attn_small_d64(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_small_d128(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_small_d256(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);

hipError_t launch_attn_small(int head_dim, bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s) {
  return head_dim == 64    ? launch_attn_small_d64(bf16, bits, p, columns, s)
         : head_dim == 128 ? launch_attn_small_d128(bf16, bits, p, columns, s)
                           : launch_attn_small_d256(bf16, bits, p, columns, s);
}

hipError_t launch_attn_tile_d64(bool bf16, int bits, const AttnParams &p, hipStream_t s);
hipError_t launch_attn_tile_d128(bool bf16, int bits, const AttnParams &p, hipStream_t s);
hipError_t launch_attn_tile_d256(bool bf16, int bits, const AttnParams &p, hipStream_t s);

hipError_t launch_attn_tile(int head_dim, bool bf16, int bits, const AttnParams &p, hipStream_t s) {
  return head_dim == 64    ? launch_attn_tile_d64(bf16, bits, p, s)
         : head_dim == 128 ? launch_attn_tile_d128(bf16, bits, p, s)
                           : launch_attn_tile_d256(bf16, bits, p, s);
}

}  // namespace exl3

extern "C" {

exl3_status exl3_rope(const exl3_rotary *r, const int32_t *positions, int32_t tokens, int32_t head_dim, int32_t dtype,
                      const exl3_rows *q, const exl3_rows *q_out, const exl3_rows *k, const exl3_rows *k_out,
                      void *stream) {
  exl3::host_clear_error();
  exl3_status st;
  if ((st = check_shape(tokens, head_dim, dtype)) != EXL3_OK) return st;
  if ((st = check_rotary(r, positions, tokens, head_dim)) != EXL3_OK) return st;
  if ((st = check_rows(q, "q", tokens, head_dim, false)) != EXL3_OK) return st;
  if ((st = check_rows(q_out, "q_out", tokens, head_dim, true)) != EXL3_OK) return st;
  if ((st = check_in_place(q, q_out, "q_out")) != EXL3_OK) return st;
  if ((k == nullptr) != (k_out == nullptr))
    return host_fail(EXL3_ERR_INVALID_ARG, "k and k_out must be given together");
  if (k != nullptr) {
    if ((st = check_rows(k, "k", tokens, head_dim, false)) != EXL3_OK) return st;
    if ((st = check_rows(k_out, "k_out", tokens, head_dim, true)) != EXL3_OK) return st;
    if ((st = check_in_place(k, k_out, "k_out")) != EXL3_OK) return st;
  }
  if ((st = check_launch_rows(tokens, q->heads + (k ? k->heads : 0))) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  exl3::RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.q = rows_of(q);
  p.q_out = rows_of(q_out);
  p.hq = q->heads;
  if (k != nullptr) {
    p.k = rows_of(k);
    p.k_out = rows_of(k_out);
    p.hk = k->heads;
  }
  p.table = r->table;
  p.positions = positions;
  p.n_positions = r->positions;
  p.rot = r->rot;
  p.interleaved = r->interleaved;
  p.tokens = tokens;
  return launched(exl3::launch_rows(head_dim, dtype == EXL3_BF16, 0, p, (hipStream_t)stream), "rope launch");
}

exl3_status exl3_cache_write(const exl3_kv_cache *c, const exl3_rows *k, const exl3_rows *v, const int32_t *slots,
                             int32_t tokens, void *stream) {
  exl3::host_clear_error();
  exl3_status st;
  if ((st = check_cache(c)) != EXL3_OK) return st;
  if ((st = check_shape(tokens, c->head_dim, c->dtype)) != EXL3_OK) return st;
  if ((st = check_rows(k, "k", tokens, c->head_dim, false)) != EXL3_OK) return st;
  if ((st = check_rows(v, "v", tokens, c->head_dim, false)) != EXL3_OK) return st;
  if (k->heads != c->heads || v->heads != c->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "k has %d heads, v %d, the cache %d", k->heads, v->heads, c->heads);
  if ((st = check_launch_rows(tokens, 2 * (int64_t)c->heads)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if ((st = check_ints(slots, "slots")) != EXL3_OK) return st;
  exl3::RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.k = rows_of(k);
  p.v = rows_of(v);
  p.hk = p.hv = c->heads;
  p.slots = slots;
  p.tokens = tokens;
  p.cache = view_of(c);
  return launched(exl3::launch_rows(c->head_dim, c->dtype == EXL3_BF16, c->bits, p, (hipStream_t)stream),
                  "cache write launch");
}

exl3_status exl3_rope_cache_write(const exl3_kv_cache *c, const exl3_rotary *r, const int32_t *positions,
                                  const int32_t *slots, int32_t tokens, const exl3_rows *q, const exl3_rows *q_out,
                                  const exl3_rows *k, const exl3_rows *k_out, const exl3_rows *v, void *stream) {
  exl3::host_clear_error();
  exl3_status st;
  if ((st = check_cache(c)) != EXL3_OK) return st;
  const int32_t D = c->head_dim;
  if ((st = check_shape(tokens, D, c->dtype)) != EXL3_OK) return st;
  if ((st = check_rotary(r, positions, tokens, D)) != EXL3_OK) return st;
  if ((st = check_rows(q, "q", tokens, D, false)) != EXL3_OK) return st;
  if ((st = check_rows(q_out, "q_out", tokens, D, true)) != EXL3_OK) return st;
  if ((st = check_in_place(q, q_out, "q_out")) != EXL3_OK) return st;
  if ((st = check_rows(k, "k", tokens, D, false)) != EXL3_OK) return st;
  if (k_out != nullptr) {
    if ((st = check_rows(k_out, "k_out", tokens, D, true)) != EXL3_OK) return st;
    if ((st = check_in_place(k, k_out, "k_out")) != EXL3_OK) return st;
  }
  if ((st = check_rows(v, "v", tokens, D, false)) != EXL3_OK) return st;
  if (k->heads != c->heads || v->heads != c->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "k has %d heads, v %d, the cache %d", k->heads, v->heads, c->heads);
  if ((st = check_launch_rows(tokens, q->heads + 2 * (int64_t)c->heads)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if ((st = check_ints(slots, "slots")) != EXL3_OK) return st;
  exl3::RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.q = rows_of(q);
  p.q_out = rows_of(q_out);
  p.k = rows_of(k);
  if (k_out != nullptr) p.k_out = rows_of(k_out);
  p.v = rows_of(v);
  p.hq = q->heads;
  p.hk = p.hv = c->heads;
  p.table = r->table;
  p.positions = positions;
  p.slots = slots;
  p.n_positions = r->positions;
  p.rot = r->rot;
  p.interleaved = r->interleaved;
  p.tokens = tokens;
  p.cache = view_of(c);
  return launched(exl3::launch_rows(D, c->dtype == EXL3_BF16, c->bits, p, (hipStream_t)stream),
                  "rope and cache write launch");
}

exl3_status exl3_cache_read(const exl3_kv_cache *c, const int32_t *slots, int32_t n, const exl3_rows *k_out,
                            const exl3_rows *v_out, void *stream) {
  exl3::host_clear_error();
  exl3_status st;
  if ((st = check_cache(c)) != EXL3_OK) return st;
  if ((st = check_shape(n, c->head_dim, c->dtype)) != EXL3_OK) return st;
  if ((st = check_rows(k_out, "k_out", n, c->head_dim, true)) != EXL3_OK) return st;
  if ((st = check_rows(v_out, "v_out", n, c->head_dim, true)) != EXL3_OK) return st;
  if (k_out->heads != c->heads || v_out->heads != c->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "k_out has %d heads, v_out %d, the cache %d", k_out->heads, v_out->heads,
                     c->heads);
  if ((st = check_launch_rows(n, 2 * (int64_t)c->heads)) != EXL3_OK) return st;
  if (n == 0) return EXL3_OK;
  if ((st = check_ints(slots, "slots")) != EXL3_OK) return st;
  exl3::ReadParams p;
  std::memset(&p, 0, sizeof p);
  p.k_out = rows_of(k_out);
  p.v_out = rows_of(v_out);
  p.slots = slots;
  p.n = n;
  p.cache = view_of(c);
  return launched(exl3::launch_cache_read(c->head_dim, c->dtype == EXL3_BF16, c->bits, p, (hipStream_t)stream),
                  "cache read launch");
}

size_t exl3_attention_workspace_bytes(int32_t batch, int32_t tokens, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim) {
  exl3::host_clear_error();
  AttnPlan pl;
  if (check_shape(tokens, head_dim, EXL3_BF16) != EXL3_OK) return 0;
  if (check_attention_sizes(batch, tokens, q_heads, kv_heads) != EXL3_OK) return 0;
  if (plan_attention(batch, tokens, q_heads, kv_heads, head_dim, &pl) != EXL3_OK) return 0;
  return pl.workspace;
}

exl3_status exl3_paged_attention(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out, const int32_t *cu_q,
                                 const int32_t *kv_len, const int32_t *page_table, int64_t page_table_stride,
                                 int32_t page_table_width, int32_t batch, int32_t tokens, float scale, int32_t window,
                                 void *workspace, size_t workspace_bytes, void *stream) {
  exl3::host_clear_error();
  exl3::AttnParams p;
  const exl3_status st = paged_params(p, c, q, out, cu_q, kv_len, page_table, page_table_stride, page_table_width,
                                      batch, tokens, scale, window);
  if (st != EXL3_OK || tokens == 0) return st;
  return run_plain(p, c->head_dim, c->dtype == EXL3_BF16, c->bits, q->heads, workspace, workspace_bytes,
                   (hipStream_t)stream);
}

exl3_status exl3_prompt_attention(const exl3_rows *q, const exl3_rows *k, const exl3_rows *v, const exl3_rows *out,
                                  const int32_t *cu, int32_t batch, int32_t tokens, int32_t head_dim, int32_t dtype,
                                  int32_t causal, int32_t window, float scale, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  exl3::host_clear_error();
  exl3::AttnParams p;
  const exl3_status st =
      prompt_params(p, q, k, v, out, cu, batch, tokens, head_dim, dtype, causal, window, scale);
  if (st != EXL3_OK || tokens == 0) return st;
  return run_plain(p, head_dim, dtype == EXL3_BF16, 0, q->heads, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
