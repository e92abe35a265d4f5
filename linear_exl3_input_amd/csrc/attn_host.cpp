// Host side of the C ABI declared in include/exl3_attn.h: argument checks,
// the choice of kernel, and launches.  Every check runs before any HIP call.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/exl3_attn.h"
#include "attn_launch.hpp"
#include "exl3_host.hpp"

namespace {

using exl3::host_fail;

constexpr int32_t MAX_TOKENS = 1 << 20;
constexpr int32_t MAX_HEADS = 1024;
constexpr int32_t MAX_BATCH = 1 << 16;
constexpr int32_t MAX_WINDOW = 1 << 30;  // a position minus a window fits 32 bits
constexpr int64_t MAX_GRID = 0x7FFFFFFF;

exl3_status check_ptr(const void *p, const char *name) {
  if (p == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "%s=%p is not 16-byte aligned", name, p);
  return EXL3_OK;
}

// int32 arrays need only their own alignment.
exl3_status check_ints(const void *p, const char *name) {
  if (p == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "%s=%p is not 4-byte aligned", name, p);
  return EXL3_OK;
}

exl3_status check_shape(int32_t tokens, int32_t head_dim, int32_t dtype) {
  if (tokens < 0) return host_fail(EXL3_ERR_INVALID_ARG, "tokens=%d is negative", tokens);
  if (tokens > MAX_TOKENS)
    return host_fail(EXL3_ERR_UNSUPPORTED, "tokens=%d exceeds the supported %d", tokens, MAX_TOKENS);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return host_fail(EXL3_ERR_UNSUPPORTED, "head_dim=%d, must be 64, 128 or 256", head_dim);
  if (dtype != EXL3_F16 && dtype != EXL3_BF16)
    return host_fail(EXL3_ERR_INVALID_ARG, "dtype=%d, must be 0 (fp16) or 1 (bf16)", dtype);
  return EXL3_OK;
}

exl3_status check_rows(const exl3_rows *r, const char *name, int32_t tokens, int32_t head_dim, bool output) {
  if (r == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "%s is NULL", name);
  if (r->heads < 1 || r->heads > MAX_HEADS)
    return host_fail(EXL3_ERR_INVALID_ARG, "%s has %d heads, must be 1..%d", name, r->heads, MAX_HEADS);
  if (tokens == 0) return EXL3_OK;
  exl3_status st;
  if ((st = check_ptr(r->data, name)) != EXL3_OK) return st;
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride % 8 != 0 || r->head_stride % 8 != 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "%s strides (%lld, %lld) must be non-negative multiples of 8 elements", name,
                     (long long)r->token_stride, (long long)r->head_stride);
  if (r->token_stride > (1ll << 40) || r->head_stride > (1ll << 40))
    return host_fail(EXL3_ERR_UNSUPPORTED, "%s strides (%lld, %lld) exceed 2^40 elements", name,
                     (long long)r->token_stride, (long long)r->head_stride);
  if (output) {
    // two rows of an output must not share elements
    const int64_t heads = (int64_t)(r->heads - 1) * r->head_stride + head_dim;
    const int64_t toks = (int64_t)(tokens - 1) * r->token_stride + head_dim;
    const bool heads_inside = (r->heads == 1 || r->head_stride >= head_dim) && (tokens == 1 || r->token_stride >= heads);
    const bool tokens_inside = (tokens == 1 || r->token_stride >= head_dim) && (r->heads == 1 || r->head_stride >= toks);
    if (!heads_inside && !tokens_inside)
      return host_fail(EXL3_ERR_INVALID_ARG, "%s strides (%lld, %lld): rows of %d tokens and %d heads overlap", name,
                       (long long)r->token_stride, (long long)r->head_stride, tokens, r->heads);
  }
  return EXL3_OK;
}

exl3_status check_cache(const exl3_kv_cache *c) {
  if (c == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "cache is NULL");
  exl3_status st;
  if ((st = check_shape(0, c->head_dim, c->dtype)) != EXL3_OK) return st;
  if (c->bits != 16 && c->bits != 8 && c->bits != 4)
    return host_fail(EXL3_ERR_INVALID_ARG, "cache bits=%d, must be 16, 8 or 4", c->bits);
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "page_size=%d, must be a power of two, 16..1024", c->page_size);
  if (c->pages < 1 || (int64_t)c->pages * c->page_size > 0x7FFFFFFFll)
    return host_fail(EXL3_ERR_INVALID_ARG, "%d pages of %d tokens, must be 1..2^31-1 tokens", c->pages, c->page_size);
  if (c->heads < 1 || c->heads > MAX_HEADS)
    return host_fail(EXL3_ERR_INVALID_ARG, "cache has %d heads, must be 1..%d", c->heads, MAX_HEADS);
  const int64_t page = (int64_t)c->heads * c->page_size * c->head_dim * c->bits / 8;
  const int64_t scales = (int64_t)c->heads * c->page_size * (c->head_dim / 32);
  auto stride = [&](int64_t s, int64_t least, const char *name) {
    if (s % 16 != 0 || s < least || s > (1ll << 40))
      return host_fail(EXL3_ERR_INVALID_ARG, "%s=%lld, must be a multiple of 16 of at least %lld", name, (long long)s,
                       (long long)least);
    return EXL3_OK;
  };
  if ((st = check_ptr(c->k, "cache k")) != EXL3_OK) return st;
  if ((st = check_ptr(c->v, "cache v")) != EXL3_OK) return st;
  if ((st = stride(c->k_page_bytes, page, "k_page_bytes")) != EXL3_OK) return st;
  if ((st = stride(c->v_page_bytes, page, "v_page_bytes")) != EXL3_OK) return st;
  if (c->bits != 16) {
    if ((st = check_ptr(c->k_scale, "cache k_scale")) != EXL3_OK) return st;
    if ((st = check_ptr(c->v_scale, "cache v_scale")) != EXL3_OK) return st;
    if ((st = stride(c->k_scale_page_bytes, scales, "k_scale_page_bytes")) != EXL3_OK) return st;
    if ((st = stride(c->v_scale_page_bytes, scales, "v_scale_page_bytes")) != EXL3_OK) return st;
  } else if (c->k_scale != nullptr || c->v_scale != nullptr) {
    return host_fail(EXL3_ERR_INVALID_ARG, "a 16-bit cache has no scales");
  }
  return EXL3_OK;
}

exl3_status check_rotary(const exl3_rotary *r, const int32_t *positions, int32_t tokens, int32_t head_dim) {
  if (r == nullptr) return host_fail(EXL3_ERR_INVALID_ARG, "rotary is NULL");
  exl3_status st;
  if ((st = check_ptr(r->table, "rotary table")) != EXL3_OK) return st;
  if (r->positions < 1) return host_fail(EXL3_ERR_INVALID_ARG, "rotary has %d positions", r->positions);
  if (r->rot < 16 || r->rot % 16 != 0 || r->rot > head_dim)
    return host_fail(EXL3_ERR_INVALID_ARG, "rot=%d, must be a multiple of 16 up to head_dim=%d", r->rot, head_dim);
  if (r->interleaved != 0 && r->interleaved != 1)
    return host_fail(EXL3_ERR_INVALID_ARG, "interleaved=%d, must be 0 or 1", r->interleaved);
  return tokens == 0 ? EXL3_OK : check_ints(positions, "positions");
}

// An output that starts where its input does is that input, in place.
exl3_status check_in_place(const exl3_rows *in, const exl3_rows *out, const char *name) {
  if (in->heads != out->heads)
    return host_fail(EXL3_ERR_INVALID_ARG, "%s has %d heads, its input %d", name, out->heads, in->heads);
  if (in->data == out->data && (in->token_stride != out->token_stride || in->head_stride != out->head_stride))
    return host_fail(EXL3_ERR_INVALID_ARG, "%s starts at its input with other strides", name);
  return EXL3_OK;
}

exl3_status check_launch_rows(int64_t tokens, int64_t heads) {
  if (tokens * heads >= (1ll << 31))
    return host_fail(EXL3_ERR_UNSUPPORTED, "%lld tokens x %lld heads exceed 2^31 rows", (long long)tokens,
                     (long long)heads);
  return EXL3_OK;
}

exl3::Rows rows_of(const exl3_rows *r) {
  return {static_cast<uint16_t *>(r->data), r->token_stride, r->head_stride};
}

exl3::CacheView view_of(const exl3_kv_cache *c) {
  exl3::CacheView v;
  std::memset(&v, 0, sizeof v);
  v.k = static_cast<uint8_t *>(c->k);
  v.v = static_cast<uint8_t *>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.k_page = c->k_page_bytes;
  v.v_page = c->v_page_bytes;
  v.ks_page = c->k_scale_page_bytes;
  v.vs_page = c->v_scale_page_bytes;
  v.pages = c->pages;
  v.page_shift = __builtin_ctz((unsigned)c->page_size);
  v.heads = c->heads;
  return v;
}

exl3_status launched(hipError_t e, const char *what) {
  return e == hipSuccess ? EXL3_OK : host_fail(EXL3_ERR_LAUNCH, "%s: %s", what, hipGetErrorString(e));
}

// ------------------------------------------------------------ attention

struct AttnPlan {
  int32_t columns;  // 16-row column tiles of a workgroup of the small kernel; 0: the tile kernel
  int32_t target;   // work items per head that splitting aims at; 0: keys are not split
  int32_t part_min, part_cap;
  size_t workspace;
};

// Splitting aims at a multiple of a round, one or two workgroups on every CU
// (find_work).  Few tiles split into equal parts, and one round is best (3
// sequences of up to 120000 keys, 4 bits, heads of 256: 96 us in one round,
// 111 in two, 136 in four); tiles of unequal keys need more, smaller parts to
// even out (64 sequences of up to 16000 keys, 8 bits: 242 us in one round, 190
// in two, 201 in four; chunks of up to 1000 tokens over 20000 keys on the tile
// kernel: 890, 803 and 712 us in one, two and four).
//
// The workgroups that a round counts on a CU are a choice, not what an
// instance's registers allow: of the small kernel two fit with heads of 256 at
// 4 bits, where one is counted, and three with most of the narrower heads,
// where two are.  Counted as they fit, those calls' times fall by 6 to 12%, but
// the same rule then gives others twice (heads of 64: 1.5 times) the parts, and
// those take 5 to 38% more.
//
// The least keys of a part: splitting costs the write and the read of a part's
// sums, 8 KB (heads of 128) in the small kernel, 66 KB in the tile kernel (132
// KB with heads of 256).  One token over 1100 keys takes 10.3 us in parts of 128
// keys at least, 9.4 in parts of 256, 10.7 in parts of 384 and 12.2 in parts of
// 1024.  On the tile kernel prompts of up to 300 tokens take 23 us split in two
// and 14 us whole, 16 sequences of 8 tokens over 4000 keys (24/4 heads of 256)
// 347 us in parts of 256 and 100 in parts of 1024, 16 of 16 tokens (32/8 heads
// of 128) 74 us in parts of 512 and 57 in parts of 1024.
constexpr int32_t PART_MIN = 256;
constexpr int32_t TILE_PART_MIN = 1024;

// A sequence's rows on one key/value head above which the tile kernel runs.
// Measured small / tile: heads of 64, 16 sequences of 4000 keys, 64 rows 43 /
// 37 us; heads of 128, 32 rows 51 / 53, 64 rows 61 / 57 (one sequence of 30000
// keys 39 / 43), 96 rows 87 / 62 (61 / 43); heads of 256, 48 rows 118 / 100, 96
// rows 167 / 104, but two sequences of 30000 keys, 96 rows, 87 / 171: few tiles
// of them need many parts, whose sums are large.
double tile_min_rows(int32_t batch, int32_t kv_heads, int32_t head_dim) {
  if (head_dim == 64) return 48.0;
  if (head_dim == 128) return 64.0;
  return 8 * (int64_t)batch * kv_heads <= exl3::host_cus() ? 128.0 : 32.0;
}

exl3_status check_attention_sizes(int32_t batch, int32_t tokens, int32_t q_heads, int32_t kv_heads) {
  if (batch < 0 || batch > MAX_BATCH)
    return host_fail(EXL3_ERR_INVALID_ARG, "batch=%d, must be 0..%d", batch, MAX_BATCH);
  if (kv_heads < 1 || q_heads < 1 || q_heads > MAX_HEADS || q_heads % kv_heads != 0)
    return host_fail(EXL3_ERR_INVALID_ARG, "%d query heads must be a multiple of the %d key/value heads, at most %d",
                     q_heads, kv_heads, MAX_HEADS);
  return EXL3_OK;
}

// The kernel and the split of a call, from its sizes alone.
exl3_status plan_attention(int32_t batch, int32_t tokens, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                           AttnPlan *pl) {
  const int32_t group = q_heads / kv_heads;
  const double rows = batch > 0 ? (double)tokens * group / batch : 0.0;  // a sequence's, on one key/value head
  pl->columns = rows > tile_min_rows(batch, kv_heads, head_dim) ? 0 : rows > 16.0 && head_dim < 256 ? 2 : 1;
  pl->target = 0;
  pl->workspace = 0;
  const bool tile = pl->columns == 0;
  pl->part_min = tile ? TILE_PART_MIN : PART_MIN;
  const int32_t R = tile ? exl3::ATTN_TILE_ROWS : 16 * pl->columns;
  const int64_t tiles = (int64_t)tokens * group / R + batch;  // at most, on each key/value head
  const int64_t per_cu = (tile ? head_dim == 256 : head_dim * pl->columns >= 256) ? 1 : 2;  // workgroups of a round
  const int64_t round = per_cu * exl3::host_cus();
  const int64_t rounds = 4 * tiles * kv_heads <= round ? 1 : tile ? 4 : 2;
  const int64_t want = std::max<int64_t>(kv_heads, rounds * round);
  pl->part_cap = 0;
  const int64_t parts = std::min(2 * (want / kv_heads), want / kv_heads + tiles);
  if (tiles * kv_heads < want && parts * kv_heads <= EXL3_WORKSPACE_COUNTER_BYTES / 4) {
    pl->target = (int32_t)(want / kv_heads);
    pl->part_cap = (int32_t)parts;
    pl->workspace = EXL3_WORKSPACE_COUNTER_BYTES + (size_t)parts * kv_heads * R * (head_dim + 2) * sizeof(float);
  }
  const int64_t items = tiles + pl->target;
  if (items * kv_heads > MAX_GRID)
    return host_fail(EXL3_ERR_UNSUPPORTED, "%d tokens x %d heads: more tiles than a launch holds", tokens, q_heads);
  return EXL3_OK;
}

exl3_status run_attention(exl3::AttnParams &p, int32_t head_dim, bool bf16, int32_t bits, int32_t q_heads,
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
  const hipError_t e = pl.columns > 0 ? exl3::launch_attn_small(head_dim, bf16, bits, p, pl.columns, s)
                                      : exl3::launch_attn_tile(head_dim, bf16, bits, p, s);
  return launched(e, "attention launch");
}

exl3_status check_scale(float scale) {
  if (!(scale > 0.f) || !std::isfinite(scale))
    return host_fail(EXL3_ERR_INVALID_ARG, "scale=%g, must be positive and finite", (double)scale);
  return EXL3_OK;
}

constexpr float LOG2E = 1.4426950408889634f;

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
