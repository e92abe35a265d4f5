// Host-side launch interface between the attention C ABI (attn_host.cpp) and
// its kernels.  Plain structs of device pointers and sizes; everything in
// them has been checked on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace exl3 {

// Division of 0 <= n < 2^31 by a number fixed on the host: with
// 2^(L-1) < d <= 2^L, n / d = (n * (2^(31+L) / d + 1)) >> (31 + L), whose
// multiplier fits 32 bits (its excess over 2^(31+L)/d is less than 1, and
// n / 2^(31+L) < 1 / d).  A device division takes about 30 instructions.
struct Divisor {
  uint32_t mul;   // 0: d is 1
  int32_t shift;  // L - 1
  static Divisor of(uint32_t d) {
    int L = 0;
    while ((1ull << L) < d) ++L;
    return d == 1 ? Divisor{0u, 0} : Divisor{(uint32_t)((1ull << (31 + L)) / d + 1), L - 1};
  }
};

// A launch has fewer than 2^32 threads along x, so workgroups (of 256) past 2^23
// go on along y.  The last row of that grid can have some too many.
constexpr int GRID_X_LOG2 = 23;
inline dim3 grid_of(int64_t workgroups) {
  const int64_t most = 1ll << GRID_X_LOG2;
  return workgroups <= most ? dim3((unsigned)workgroups)
                            : dim3((unsigned)most, (unsigned)((workgroups + most - 1) >> GRID_X_LOG2));
}

// Strided rows of 16-bit values; strides in elements.
struct Rows {
  uint16_t *data;
  int64_t token, head;
};

// The paged cache; strides in bytes.
struct CacheView {
  uint8_t *k, *v;
  uint8_t *k_scale, *v_scale;
  int64_t k_page, v_page, ks_page, vs_page;
  int32_t pages, page_shift, heads;
};

// Rotation and cache write of one launch: per token hq + hk + hv rows.
struct RowsParams {
  Rows q, q_out, k, k_out, v;  // k_out.data null: not written
  int32_t hq, hk, hv;          // hv > 0: k and v go to the cache
  const float *table;          // null: no rotation (q unused)
  const int32_t *positions;
  const int32_t *slots;
  int32_t n_positions, rot, interleaved;
  int32_t tokens;
  CacheView cache;
};

struct ReadParams {
  Rows k_out, v_out;
  const int32_t *slots;
  int32_t n;
  CacheView cache;
};

// Keys of a sequence that the kernels address; positions past them, and steps
// that run a little past a sequence's end, still fit 32 bits.
constexpr int32_t MAX_KEYS = 0x7FFF0000;

// Attention over a paged cache (cache.k set) or packed rows (k.data set).
struct AttnParams {
  Rows q, out, k, v;
  CacheView cache;
  const int32_t *cu;          // [batch+1] query rows of each sequence
  const int32_t *kv_len;      // paged: keys of each sequence
  const int32_t *page_table;
  int64_t table_stride;
  int32_t table_width;
  int32_t table_keys;         // keys that a row of the table can have (paged), at most MAX_KEYS
  int32_t batch, tokens, heads_kv, group;
  Divisor by_group;
  int32_t causal, window;     // window 0: none
  float scale_log2;           // softmax scale * log2(e)
  uint32_t *counters;         // workspace: arrivals of the split tiles
  float *part;                // workspace: partial results of the split tiles
  int32_t target;             // work items per head aimed at when keys are split (0: not split)
  int32_t part_min;           // least keys of a part
  int32_t part_cap;           // parts of a head that `part` and `counters` hold
};

// bits: 0 (no cache), 16, 8, 4.
hipError_t launch_rows(int head_dim, bool bf16, int bits, const RowsParams &p, hipStream_t s);
hipError_t launch_cache_read(int head_dim, bool bf16, int bits, const ReadParams &p, hipStream_t s);

// Tiles of 16 * columns query rows, one workgroup each (columns 1, or 2 for heads of 64 and 128).
// bits 0: packed rows.
hipError_t launch_attn_small(int head_dim, bool bf16, int bits, const AttnParams &p, int columns, hipStream_t s);
// Tiles of ATTN_TILE_ROWS query rows.
constexpr int ATTN_TILE_ROWS = 128;
hipError_t launch_attn_tile(int head_dim, bool bf16, int bits, const AttnParams &p, hipStream_t s);

}  // namespace exl3
