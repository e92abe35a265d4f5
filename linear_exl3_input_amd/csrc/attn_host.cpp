// Host side of the C ABI declared in include/exl3_attn.h: argument checks,
// the choice of kernel, and launches.  Every check runs before any HIP call.
#include "attn_checks.hpp"

namespace {

using namespace exl3;

exl3_status run_attention(AttnParams &p, int32_t head_dim, bool bf16, int32_t bits, int32_t q_heads,
                          void *workspace, size_t workspace_bytes, hipStream_t s) {
  AttnPlan pl;
  exl3_status st = plan_attention(p.batch, p.tokens, q_heads, p.heads_kv, head_dim, &pl);
  if (st != EXL3_OK) return st;
  if (pl.workspace > 0) {
    if (workspace == nullptr || workspace_bytes < pl.workspace)
      return host_fail(EXL3_ERR_WORKSPACE, "workspace of %zu bytes; this call needs %zu (short by %zu)", workspace_bytes,
                       pl.workspace, pl.workspace > workspace_bytes ? pl.workspace - workspace_bytes : (size_t)0);
    if ((st = check_ptr(workspace, "workspace")) != EXL3_OK) return st;
    p.counters = static_cast<uint32_t *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + EXL3_WORKSPACE_COUNTER_BYTES);
  }
  p.target = pl.target;
  p.part_min = pl.part_min;
  p.part_cap = pl.part_cap;
  const hipError_t e = pl.columns > 0 ? launch_attn_small(head_dim, bf16, bits, p, pl.columns, s)
                                      : launch_attn_tile(head_dim, bf16, bits, p, s);
  return launched(e, "attention launch");
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
  exl3_status st;
  if ((st = check_cache(c)) != EXL3_OK) return st;
  const int32_t D = c->head_dim;
  if ((st = check_shape(tokens, D, c->dtype)) != EXL3_OK) return st;
  if ((st = check_rows(q, "q", tokens, D, false)) != EXL3_OK) return st;
  if ((st = check_rows(out, "out", tokens, D, true)) != EXL3_OK) return st;
  if (q->heads != out->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "out has %d heads, q %d", out->heads, q->heads);
  if ((st = check_attention_sizes(batch, tokens, q->heads, c->heads)) != EXL3_OK) return st;
  if (page_table_width < 0 || page_table_stride < 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "page table width=%d stride=%lld are negative", page_table_width,
                     (long long)page_table_stride);
  if (window < 0 || window > MAX_WINDOW)
    return host_fail(EXL3_ERR_INVALID_ARG, "window=%d, must be 0 (none) to %d", window, MAX_WINDOW);
  if ((st = check_scale(scale)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if (batch == 0) return host_fail(EXL3_ERR_INVALID_ARG, "batch=0 with %d tokens", tokens);
  if ((st = check_ints(cu_q, "cu_q")) != EXL3_OK) return st;
  if ((st = check_ints(kv_len, "kv_len")) != EXL3_OK) return st;
  if (page_table_width > 0 && (st = check_ints(page_table, "page_table")) != EXL3_OK) return st;
  exl3::AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.q = rows_of(q);
  p.out = rows_of(out);
  p.cache = view_of(c);
  p.cu = cu_q;
  p.kv_len = kv_len;
  p.page_table = page_table;
  p.table_stride = page_table_stride;
  p.table_width = page_table_width;
  p.table_keys = (int32_t)std::min<int64_t>((int64_t)page_table_width * c->page_size, exl3::MAX_KEYS);
  p.batch = batch;
  p.tokens = tokens;
  p.heads_kv = c->heads;
  p.group = q->heads / c->heads;
  p.by_group = exl3::Divisor::of((uint32_t)p.group);
  p.causal = 1;
  p.window = window;
  p.scale_log2 = scale * LOG2E;
  return run_attention(p, D, c->dtype == EXL3_BF16, c->bits, q->heads, workspace, workspace_bytes,
                       (hipStream_t)stream);
}

exl3_status exl3_prompt_attention(const exl3_rows *q, const exl3_rows *k, const exl3_rows *v, const exl3_rows *out,
                                  const int32_t *cu, int32_t batch, int32_t tokens, int32_t head_dim, int32_t dtype,
                                  int32_t causal, int32_t window, float scale, void *workspace, size_t workspace_bytes,
                                  void *stream) {
  exl3::host_clear_error();
  exl3_status st;
  if ((st = check_shape(tokens, head_dim, dtype)) != EXL3_OK) return st;
  if ((st = check_rows(q, "q", tokens, head_dim, false)) != EXL3_OK) return st;
  if ((st = check_rows(k, "k", tokens, head_dim, false)) != EXL3_OK) return st;
  if ((st = check_rows(v, "v", tokens, head_dim, false)) != EXL3_OK) return st;
  if ((st = check_rows(out, "out", tokens, head_dim, true)) != EXL3_OK) return st;
  if (q->heads != out->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "out has %d heads, q %d", out->heads, q->heads);
  // tiles of up to 128 keys are addressed with 32-bit offsets
  constexpr int64_t MAX_TOKEN_STRIDE = 1 << 22;
  if (k->token_stride > MAX_TOKEN_STRIDE || v->token_stride > MAX_TOKEN_STRIDE)
    return host_fail(EXL3_ERR_UNSUPPORTED, "token strides of k (%lld) and v (%lld) must be at most %lld elements",
                     (long long)k->token_stride, (long long)v->token_stride, (long long)MAX_TOKEN_STRIDE);
  if (k->heads != v->heads) return host_fail(EXL3_ERR_INVALID_ARG, "k has %d heads, v %d", k->heads, v->heads);
  if ((st = check_attention_sizes(batch, tokens, q->heads, k->heads)) != EXL3_OK) return st;
  if (causal != 0 && causal != 1) return host_fail(EXL3_ERR_INVALID_ARG, "causal=%d, must be 0 or 1", causal);
  if (window < 0 || window > MAX_WINDOW || (window > 0 && !causal))
    return host_fail(EXL3_ERR_INVALID_ARG, "window=%d with causal=%d: 0 (none) to %d, and a window is causal", window,
                     causal, MAX_WINDOW);
  if ((st = check_scale(scale)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if (batch == 0) return host_fail(EXL3_ERR_INVALID_ARG, "batch=0 with %d tokens", tokens);
  if ((st = check_ints(cu, "cu")) != EXL3_OK) return st;
  exl3::AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.q = rows_of(q);
  p.out = rows_of(out);
  p.k = rows_of(k);
  p.v = rows_of(v);
  p.cu = cu;
  p.batch = batch;
  p.tokens = tokens;
  p.heads_kv = k->heads;
  p.group = q->heads / k->heads;
  p.by_group = exl3::Divisor::of((uint32_t)p.group);
  p.causal = causal;
  p.window = window;
  p.scale_log2 = scale * LOG2E;
  return run_attention(p, head_dim, dtype == EXL3_BF16, 0, q->heads, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
