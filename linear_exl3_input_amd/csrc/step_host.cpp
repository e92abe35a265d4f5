// Host side of the C ABI declared in include/exl3_step.h: argument checks and
// launches.  Every check runs before any HIP call.
#include "../../include/exl3_step.h"
#include "attn_checks.hpp"
#include "step_launch.hpp"

namespace {

using namespace exl3;

exl3_status check_axes(const exl3_rotary_axes *r, const int32_t *positions, int64_t axis_stride, int32_t tokens,
                       int32_t head_dim) {
  if (r == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "rotary is NULL");
  exl3_status st;
  if ((st = check_rotary(&r->rotary, positions, tokens, head_dim)) != EXL3_OK) return st;
  if (r->axes < 1 || r->axes > 4) return host_fail(EXL3_ERR_INVALID_ARG, "axes=%d, must be 1..4", r->axes);
  for (int i = 0; i < r->rotary.rot / 2; ++i) {
    const int a = (int)((r->axis_of[i / 16] >> (2 * (i % 16))) & 3u);
    if (a >= r->axes) return host_fail(EXL3_ERR_INVALID_ARG, "pair %d turns by axis %d of %d", i, a, r->axes);
  }
  if (axis_stride < 0 || axis_stride > (1ll << 40))
    return host_fail(EXL3_ERR_INVALID_ARG, "axis_stride=%lld, must be 0..2^40", (long long)axis_stride);
  return EXL3_OK;
}

exl3_status check_norm(const exl3_head_norm *n, const exl3_rows *q, const exl3_rows *k) {
  if (n == nullptr) return EXL3_OK;
  exl3_status st;
  if ((st = check_ptr(n->q, "norm q")) != EXL3_OK) return st;
  if (n->q_rows != 1 && n->q_rows != q->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "norm has weights of %d query heads, q has %d", n->q_rows, q->heads);
  if (k != nullptr) {
    if ((st = check_ptr(n->k, "norm k")) != EXL3_OK) return st;
    if (n->k_rows != 1 && n->k_rows != k->heads)
      return host_fail(EXL3_ERR_INVALID_ARG, "norm has weights of %d key heads, k has %d", n->k_rows, k->heads);
  }
  if (!(n->eps >= 1e-30f && n->eps <= 1.f))
    return host_fail(EXL3_ERR_INVALID_ARG, "eps=%g, must be 1e-30..1", (double)n->eps);
  return EXL3_OK;
}

NormRowsParams norm_rows(const exl3_rotary_axes *r, const exl3_head_norm *n, const int32_t *positions,
                         int64_t axis_stride, int32_t tokens, int32_t head_dim, const exl3_rows *q,
                         const exl3_rows *q_out, const exl3_rows *k, const exl3_rows *k_out) {
  NormRowsParams p;
  std::memset(&p, 0, sizeof p);
  p.rows.q = rows_of(q);
  p.rows.q_out = rows_of(q_out);
  p.rows.hq = q->heads;
  if (k != nullptr) {
    p.rows.k = rows_of(k);
    p.rows.hk = k->heads;
  }
  if (k_out != nullptr) p.rows.k_out = rows_of(k_out);
  p.rows.table = r->rotary.table;
  p.rows.positions = positions;
  p.rows.n_positions = r->rotary.positions;
  p.rows.rot = r->rotary.rot;
  p.rows.interleaved = r->rotary.interleaved;
  p.rows.tokens = tokens;
  p.axis_stride = axis_stride;
  std::memcpy(p.axis_of, r->axis_of, sizeof p.axis_of);
  p.axes = r->axes;
  if (n != nullptr) {
    p.wq = n->q;
    p.wk = n->k;
    p.wq_step = n->q_rows > 1 ? head_dim : 0;
    p.wk_step = n->k_rows > 1 ? head_dim : 0;
    p.eps = n->eps;
  }
  return p;
}

bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {  // ranges of int32
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && a != nullptr && b != nullptr && x < y + 4 * (uintptr_t)bn && y < x + 4 * (uintptr_t)an;
}

// Positions, sinks and windows stay within 32 bits.
constexpr int32_t MAX_SINKS = 1 << 20;

exl3_status check_sinks(int32_t sinks, int32_t window) {
  if (sinks < 0 || sinks > MAX_SINKS)
    return host_fail(EXL3_ERR_INVALID_ARG, "sinks=%d, must be 0..%d", sinks, MAX_SINKS);
  if (window < 1) return host_fail(EXL3_ERR_INVALID_ARG, "window=%d: first tokens beside a window need one", window);
  return EXL3_OK;
}

exl3_status run_sinks(AttnParams &p, int32_t head_dim, bool bf16, int32_t bits, int32_t q_heads, int32_t sinks,
                      void *workspace, size_t workspace_bytes, hipStream_t s) {
  p.sinks = sinks;
  p.sink_keys = (sinks + 127) & ~127;  // both kernels' steps are at most 128 keys
  // Where most sequences can be longer than what a row sees, all tiles have about
  // as many keys, and parts for one round of the GPU are best (32 sequences, one
  // token each, windows of 4096, 8 heads of 128: 53 us in one round, 62 in two,
  // 66 whole; 3 chunks of up to 900 tokens, windows of 2048: 100 us in one round,
  // 128 in four): less than the plain calls' rule, whose workspace so suffices.
  const int64_t keys = p.kv_len != nullptr ? p.table_keys : p.tokens / p.batch;
  const int32_t rounds = 2 * ((int64_t)p.window + sinks) <= keys ? 1 : 0;
  AttnPlan pl;
  const exl3_status st =
      plan_split(p.batch, p.tokens, q_heads, p.heads_kv, head_dim,
                 plan_columns(p.batch, p.tokens, q_heads, p.heads_kv, head_dim), &pl, rounds);
  if (st != EXL3_OK) return st;
  const WorkspaceTurn turn(pl.workspace > 0 ? workspace : nullptr);
  return run_planned(p, pl, workspace, workspace_bytes,
                     [&](int columns) { return launch_attn_sinks(head_dim, bf16, bits, p, columns, s); });
}

// The workspace of a call with shared prefixes: the counters and the own keys'
// parts, what the groups are, and the state of every part's rows.
struct PrefixPlan {
  AttnPlan shared, own;  // the groups as sequences; the sequences
  int32_t items;         // of the shared keys, at most, on each key/value head
  int32_t rows_log2;     // rows of an item
  size_t ints, state, workspace;  // offsets
  bool shares;           // else the call is paged_attention's, whatever it is given
};

// A call whose shared keys, read by every sequence for itself, are fewer bytes
// than this is paged_attention's: they come from the caches at 8 to 9 TB/s, and
// the two passes take 16 to 25 us with hardly a key.  Measured shared / plain, one
// token, 32/8 heads of 128, 8 bits: 4 sequences of 8192 and 32768 shared keys (54
// and 210 MB) 22 / 21 us and 32 / 42, 8 (126, 489) 25 / 25 and 37 / 67, 16 of 2048
// and 8192 (75, 270) 22 / 27 and 27 / 46, 64 of 512 and 2048 (111, 315) 29 / 27 and
// 32 / 47; 8 tokens each, 16 of 8192 (270) 53 / 52.  24/4 heads of 256 need more, at
// 4 bits 24 sequences of 8192 (213) 55 / 44, 32 (287) 57 / 50 and 64 (583) 66 / 87;
// 32/8 heads of 256 do not, 16 of 8192 (278) 34 / 50.  One number for all of them:
// it shares the 24 and 32 sequences of those wide heads, 11 and 7 us too slow, and
// leaves the 16 of 2048 keys plain, where later measurements found no difference
// (26 / 26; 64 of 512 25 / 25).  The host knows the page table's width alone, so
// that counts as every sequence's keys.
constexpr double SHARED_BYTES_MIN = 192e6;

// And so is a call whose sequences fill the tile kernel's tiles by themselves, for
// what every tile leaves costs more than the keys: by the average rows of a
// sequence on a key/value head, over 8192 shared and 150 own keys, 32/8 heads of 128,
// 8 bits, shared / plain, 16 sequences of 256 rows 215 / 252 us, 512 361 / 380, 1024
// 666 / 656, 2048 1275 / 1227; 64 sequences of 256 rows 671 / 657, 512 1319 / 1252, 1024
// 2598 / 2472; 24/4 heads of 256, 16 sequences of 1536 rows 1396 / 1393.
constexpr int64_t SHARED_ROWS_MAX = 512;

// And so is a call whose state would be larger than this: it grows with the query
// rows (528 bytes each with heads of 128) where the plain call's parts do not.
// What it costs: with 32 heads of 128 a call reaches it at 60000 tokens, where
// sharing 8192 keys still gains a quarter if a sequence has 64 rows on a key/value
// head (2048 sequences of 16 tokens, 593 MB, 6631 / 8890 us), and nothing if it has
// 128 and more (512 of 32 tokens, 312 MB, 2575 / 2461; 2048 of 64 tokens, 64 heads,
// 4.5 GB, 40548 / 39605).
constexpr size_t STATE_MAX = (size_t)1 << 30;

bool worth_sharing(const exl3_kv_cache *c, int32_t page_table_width, int32_t batch, int32_t groups) {
  const double row = c->head_dim * c->bits / 8.0 + (c->bits < 16 ? c->head_dim / 32.0 : 0.0);
  return groups > 0 && (double)(batch - groups) * page_table_width * c->page_size * c->heads * 2 * row >=
                           SHARED_BYTES_MIN;
}

exl3_status plan_prefix(int32_t batch, int32_t tokens, int32_t groups, int32_t q_heads, int32_t kv_heads,
                        int32_t head_dim, PrefixPlan *pl) {
  exl3_status st;
  if (groups < 0 || groups > batch)
    return host_fail(EXL3_ERR_INVALID_ARG, "groups=%d, must be 0..batch=%d", groups, batch);
  AttnPlan plain;  // a call that is not worth it
  if ((st = plan_attention(batch, tokens, q_heads, kv_heads, head_dim, &plain)) != EXL3_OK) return st;
  pl->workspace = std::max(plain.workspace, (size_t)EXL3_WORKSPACE_COUNTER_BYTES);
  pl->shares = (int64_t)tokens * (q_heads / kv_heads) <= SHARED_ROWS_MAX * batch;
  if (!pl->shares) return EXL3_OK;
  // Own keys: 16 rows a workgroup rather than 32, since each of them reads what
  // the shared keys left for its rows (16 sequences of 8 tokens, 8 heads of 128:
  // 19 us, with 32 rows 29), and in parts only where whole sequences do not
  // fill the GPU (64 sequences of up to 1500 own keys: 39 us whole, 44 in parts).
  const int32_t own = plan_columns(batch, tokens, q_heads, kv_heads, head_dim);
  st = plan_split(batch, tokens, q_heads, kv_heads, head_dim, std::min(own, 1), &pl->own);
  if (st != EXL3_OK) return st;
  if ((int64_t)batch * kv_heads >= host_cus()) {
    pl->own.target = pl->own.part_cap = 0;
    pl->own.workspace = 0;
  }
  pl->own.part_min = std::max(pl->own.part_min, 1024);
  // Shared keys: as many parts as fill the GPU once, since joining them is cheap
  // (state_row): two workgroups of the tile kernel a CU (one with heads of
  // 256), one of the small kernel.
  pl->shared.columns = plan_columns(groups, tokens, q_heads, kv_heads, head_dim);
  const bool tile = pl->shared.columns == 0;
  pl->shared.target = std::max(1, (tile && head_dim < 256 ? 2 : 1) * host_cus() / kv_heads);
  pl->shared.part_min = 256;
  pl->rows_log2 = __builtin_ctz((unsigned)tile_rows(pl->shared.columns));
  const int64_t items = ((int64_t)tokens * (q_heads / kv_heads) >> pl->rows_log2) + groups + pl->shared.target;
  const int64_t state_rows = items * kv_heads << pl->rows_log2;
  const size_t state = sizeof(float) * (size_t)state_rows * (STATE_PAD + head_dim);
  pl->shares = state <= STATE_MAX;  // (a launch holds the tiles of far larger ones)
  if (!pl->shares) return EXL3_OK;
  pl->items = (int32_t)items;
  auto whole = [](size_t n) { return (n + 255) & ~(size_t)255; };
  pl->ints = whole(std::max(pl->own.workspace, (size_t)EXL3_WORKSPACE_COUNTER_BYTES));
  pl->state = pl->ints + whole(sizeof(int32_t) * (4 * (size_t)batch + 2 + 6 * (size_t)groups + 2));
  pl->workspace = std::max(pl->workspace, pl->state + state);
  return EXL3_OK;
}

}  // namespace

namespace exl3 {

hipError_t launch_attn_prefix_d64(bool bf16, int bits, const PrefixParams &p, int columns, hipStream_t s);
hipError_t launch_attn_prefix_d128(bool bf16, int bits, const PrefixParams &p, int columns, hipStream_t s);
hipError_t launch_attn_prefix_d256(bool bf16, int bits, const PrefixParams &p, int columns, hipStream_t s);

hipError_t launch_attn_prefix(int head_dim, bool bf16, int bits, const PrefixParams &p, int columns, hipStream_t s) {
  return head_dim == 64    ? launch_attn_prefix_d64(bf16, bits, p, columns, s)
         : head_dim == 128 ? launch_attn_prefix_d128(bf16, bits, p, columns, s)
                           : launch_attn_prefix_d256(bf16, bits, p, columns, s);
}

hipError_t launch_attn_own_d64(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_own_d128(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_own_d256(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);

hipError_t launch_attn_own(int head_dim, bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s) {
  return head_dim == 64    ? launch_attn_own_d64(bf16, bits, p, columns, s)
         : head_dim == 128 ? launch_attn_own_d128(bf16, bits, p, columns, s)
                           : launch_attn_own_d256(bf16, bits, p, columns, s);
}

hipError_t launch_attn_sinks_d64(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_sinks_d128(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
hipError_t launch_attn_sinks_d256(bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);

hipError_t launch_attn_sinks(int head_dim, bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s) {
  return head_dim == 64    ? launch_attn_sinks_d64(bf16, bits, p, columns, s)
         : head_dim == 128 ? launch_attn_sinks_d128(bf16, bits, p, columns, s)
                           : launch_attn_sinks_d256(bf16, bits, p, columns, s);
}

}  // namespace exl3

extern "C" {

exl3_status exl3_norm_rope(const exl3_rotary_axes *r, const exl3_head_norm *n, const int32_t *positions,
                           int64_t axis_stride, int32_t tokens, int32_t head_dim, int32_t dtype, const exl3_rows *q,
                           const exl3_rows *q_out, const exl3_rows *k, const exl3_rows *k_out, void *stream) {
  host_clear_error();
  exl3_status st;
  if ((st = check_shape(tokens, head_dim, dtype)) != EXL3_OK) return st;
  if ((st = check_axes(r, positions, axis_stride, tokens, head_dim)) != EXL3_OK) return st;
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
  if ((st = check_norm(n, q, k)) != EXL3_OK) return st;
  if ((st = check_launch_rows(tokens, q->heads + (k ? k->heads : 0))) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  const NormRowsParams p = norm_rows(r, n, positions, axis_stride, tokens, head_dim, q, q_out, k, k_out);
  return launched(launch_norm_rows(head_dim, dtype == EXL3_BF16, 0, p, (hipStream_t)stream), "norm and rope launch");
}

exl3_status exl3_norm_rope_cache_write(const exl3_kv_cache *c, const exl3_rotary_axes *r, const exl3_head_norm *n,
                                       const int32_t *positions, int64_t axis_stride, const int32_t *slots,
                                       int32_t tokens, const exl3_rows *q, const exl3_rows *q_out, const exl3_rows *k,
                                       const exl3_rows *k_out, const exl3_rows *v, void *stream) {
  host_clear_error();
  exl3_status st;
  if ((st = check_cache(c)) != EXL3_OK) return st;
  const int32_t D = c->head_dim;
  if ((st = check_shape(tokens, D, c->dtype)) != EXL3_OK) return st;
  if ((st = check_axes(r, positions, axis_stride, tokens, D)) != EXL3_OK) return st;
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
  if ((st = check_norm(n, q, k)) != EXL3_OK) return st;
  if ((st = check_launch_rows(tokens, q->heads + 2 * (int64_t)c->heads)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if ((st = check_ints(slots, "slots")) != EXL3_OK) return st;
  NormRowsParams p = norm_rows(r, n, positions, axis_stride, tokens, D, q, q_out, k, k_out);
  p.rows.v = rows_of(v);
  p.rows.hv = c->heads;
  p.rows.slots = slots;
  p.rows.cache = view_of(c);
  return launched(launch_norm_rows(D, c->dtype == EXL3_BF16, c->bits, p, (hipStream_t)stream),
                  "norm, rope and cache write launch");
}

exl3_status exl3_cache_extend(int32_t pages, int32_t page_size, const int32_t *q_len, const int32_t *kv_len,
                              int32_t batch, int32_t *page_table, int64_t page_table_stride, int32_t page_table_width,
                              const int32_t *free_pages, int32_t n_free, const int32_t *taken, int32_t tokens,
                              int32_t *cu_q, int32_t *kv_out, int32_t *positions, int32_t *slots, int32_t *counts,
                              void *stream) {
  host_clear_error();
  exl3_status st;
  if ((st = check_pages(pages, page_size)) != EXL3_OK) return st;
  if (batch < 0 || batch > MAX_BATCH)
    return host_fail(EXL3_ERR_INVALID_ARG, "batch=%d, must be 0..%d", batch, MAX_BATCH);
  if (tokens < 0 || tokens > MAX_TOKENS)
    return host_fail(EXL3_ERR_INVALID_ARG, "tokens=%d, must be 0..%d", tokens, MAX_TOKENS);
  if (n_free < 0) return host_fail(EXL3_ERR_INVALID_ARG, "n_free=%d is negative", n_free);
  if (page_table_width < 0 || (batch > 1 && page_table_stride < page_table_width))
    return host_fail(EXL3_ERR_INVALID_ARG, "page table width=%d stride=%lld: rows of %d entries overlap",
                     page_table_width, (long long)page_table_stride, page_table_width);
  if (page_table_stride < 0 || page_table_stride > (1ll << 40))
    return host_fail(EXL3_ERR_INVALID_ARG, "page table stride=%lld, must be 0..2^40", (long long)page_table_stride);
  const int64_t entries = batch > 0 && page_table_width > 0 ? (int64_t)(batch - 1) * page_table_stride + page_table_width : 0;
  struct Array {
    const void *data;
    int64_t n;
    const char *name;
    bool output;
  };
  const Array arrays[] = {{q_len, batch, "q_len", false},
                          {kv_len, batch, "kv_len", false},
                          {free_pages, n_free, "free_pages", false},
                          {taken, taken != nullptr, "taken", false},
                          {page_table, entries, "page_table", true},
                          {cu_q, batch + 1, "cu_q", true},
                          {kv_out, batch, "kv_out", true},
                          {positions, tokens, "positions", true},
                          {slots, tokens, "slots", true},
                          {counts, 2, "counts", true}};
  for (const Array &a : arrays)
    if (a.n > 0 && (st = check_ints(a.data, a.name)) != EXL3_OK) return st;
  for (const Array &a : arrays)
    for (const Array &b : arrays)
      if (&a < &b && (a.output || b.output) && overlap(a.data, a.n, b.data, b.n))
        return host_fail(EXL3_ERR_INVALID_ARG, "%s and %s overlap", a.name, b.name);
  TablesParams p;
  std::memset(&p, 0, sizeof p);
  p.q_len = q_len;
  p.kv_len = kv_len;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.free_pages = free_pages;
  p.taken = taken;
  p.cu = cu_q;
  p.kv_out = kv_out;
  p.positions = positions;
  p.slots = slots;
  p.counts = counts;
  p.batch = batch;
  p.tokens = tokens;
  p.width = page_table_width;
  p.pages = pages;
  p.page_shift = __builtin_ctz((unsigned)page_size);
  p.n_free = n_free;
  return launched(launch_tables(p, (hipStream_t)stream), "table launch");
}

exl3_status exl3_paged_attention_sinks(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out,
                                       const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                                       int64_t page_table_stride, int32_t page_table_width, int32_t batch,
                                       int32_t tokens, float scale, int32_t window, int32_t sinks, void *workspace,
                                       size_t workspace_bytes, void *stream) {
  host_clear_error();
  AttnParams p;
  exl3_status st;
  if ((st = check_sinks(sinks, window)) != EXL3_OK) return st;
  st = paged_params(p, c, q, out, cu_q, kv_len, page_table, page_table_stride, page_table_width, batch, tokens, scale,
                    window);
  if (st != EXL3_OK || tokens == 0) return st;
  return run_sinks(p, c->head_dim, c->dtype == EXL3_BF16, c->bits, q->heads, sinks, workspace, workspace_bytes,
                   (hipStream_t)stream);
}

exl3_status exl3_prompt_attention_sinks(const exl3_rows *q, const exl3_rows *k, const exl3_rows *v,
                                        const exl3_rows *out, const int32_t *cu, int32_t batch, int32_t tokens,
                                        int32_t head_dim, int32_t dtype, int32_t window, int32_t sinks, float scale,
                                        void *workspace, size_t workspace_bytes, void *stream) {
  host_clear_error();
  AttnParams p;
  exl3_status st;
  if ((st = check_sinks(sinks, window)) != EXL3_OK) return st;
  st = prompt_params(p, q, k, v, out, cu, batch, tokens, head_dim, dtype, 1, window, scale);
  if (st != EXL3_OK || tokens == 0) return st;
  return run_sinks(p, head_dim, dtype == EXL3_BF16, 0, q->heads, sinks, workspace, workspace_bytes,
                   (hipStream_t)stream);
}

size_t exl3_prefix_attention_workspace_bytes(int32_t batch, int32_t tokens, int32_t groups, int32_t q_heads,
                                             int32_t kv_heads, int32_t head_dim) {
  host_clear_error();
  PrefixPlan pl;
  if (check_shape(tokens, head_dim, EXL3_BF16) != EXL3_OK) return 0;
  if (check_attention_sizes(batch, tokens, q_heads, kv_heads) != EXL3_OK) return 0;
  if (plan_prefix(batch, tokens, groups, q_heads, kv_heads, head_dim, &pl) != EXL3_OK) return 0;
  return pl.workspace;
}

exl3_status exl3_prefix_attention(const exl3_kv_cache *c, const exl3_rows *q, const exl3_rows *out,
                                  const int32_t *cu_q, const int32_t *kv_len, const int32_t *page_table,
                                  int64_t page_table_stride, int32_t page_table_width, int32_t batch, int32_t tokens,
                                  const int32_t *group_cu, const int32_t *prefix_len, int32_t groups, float scale,
                                  void *workspace, size_t workspace_bytes, void *stream) {
  host_clear_error();
  AttnParams p;
  exl3_status st = paged_params(p, c, q, out, cu_q, kv_len, page_table, page_table_stride, page_table_width, batch,
                                tokens, scale, 0);
  if (st != EXL3_OK) return st;
  const int32_t D = c->head_dim;
  PrefixPlan pl;
  if ((st = plan_prefix(batch, tokens, groups, q->heads, c->heads, D, &pl)) != EXL3_OK) return st;
  if (tokens == 0) return EXL3_OK;
  if ((st = check_ints(group_cu, "group_cu")) != EXL3_OK) return st;
  if (groups > 0 && (st = check_ints(prefix_len, "prefix_len")) != EXL3_OK) return st;
  if (workspace == nullptr || workspace_bytes < pl.workspace)
    return host_fail(EXL3_ERR_WORKSPACE, "workspace of %zu bytes; this call needs %zu (short by %zu)", workspace_bytes,
                     pl.workspace, pl.workspace > workspace_bytes ? pl.workspace - workspace_bytes : (size_t)0);
  if ((st = check_ptr(workspace, "workspace")) != EXL3_OK) return st;
  if (!pl.shares || !worth_sharing(c, page_table_width, batch, groups))
    return exl3_paged_attention(c, q, out, cu_q, kv_len, page_table, page_table_stride, page_table_width, batch, tokens,
                                scale, 0, workspace, workspace_bytes, stream);
  const hipStream_t s = (hipStream_t)stream;
  const bool bf16 = c->dtype == EXL3_BF16;
  char *ws = static_cast<char *>(workspace);
  int32_t *ints = reinterpret_cast<int32_t *>(ws + pl.ints);
  auto take = [&](int64_t n) {
    int32_t *at = ints;
    ints += n;
    return at;
  };
  GroupsParams g;
  std::memset(&g, 0, sizeof g);
  g.cu = cu_q;
  g.kv_len = kv_len;
  g.group_cu = group_cu;
  g.prefix_len = prefix_len;
  g.batch = batch;
  g.tokens = tokens;
  g.groups = groups;
  g.table_keys = p.table_keys;
  g.seq_row = take(batch + 1);
  g.start = take(batch);
  g.of = take(batch);
  g.first = take(groups + 1);
  g.row = take(groups + 1);
  g.keys = take(groups);
  g.lead = take(groups);
  g.tile_at = take(batch + 1);
  g.group = p.group;
  g.tile_rows = tile_rows(pl.own.columns);
  p.group_items = take(2 * (int64_t)groups);
  const WorkspaceTurn turn(workspace);
  if (batch >= FEW_SEQUENCES && (st = launched(launch_groups(g, s), "groups launch")) != EXL3_OK) return st;
  p.state = reinterpret_cast<float *>(ws + pl.state);
  PrefixParams shared;
  static_cast<AttnParams &>(shared) = p;
  shared.groups = g;
  shared.cu = g.row;
  shared.kv_len = g.keys;
  shared.table_row = g.lead;
  shared.batch = groups;
  shared.causal = 0;
  shared.target = pl.shared.target;
  shared.part_min = pl.shared.part_min;
  shared.part_cap = pl.items;
  st = launched(launch_attn_prefix(D, bf16, c->bits, shared, pl.shared.columns, s), "shared keys launch");
  if (st != EXL3_OK) return st;
  if (batch >= FEW_SEQUENCES && pl.own.target == 0) p.tile_at = g.tile_at, p.seq_row = g.seq_row;
  p.start = g.start;
  p.group_of = g.of;
  p.group_row = g.row;
  p.state_shift = pl.rows_log2;
  p.state_items = pl.items;
  return run_planned(p, pl.own, workspace, workspace_bytes,
                     [&](int columns) { return launch_attn_own(D, bf16, c->bits, p, columns, s); });
}

}  // extern "C"
