// Which keys a workgroup of the attention kernels reads: plain arithmetic, so
// that it can be checked without a GPU.
#pragma once

#include "attn_launch.hpp"

#define EXL3_BOTH __host__ __device__ __forceinline__

namespace exl3 {

template <class T>
EXL3_BOTH T least(T a, T b) { return a < b ? a : b; }
template <class T>
EXL3_BOTH T most(T a, T b) { return a > b ? a : b; }

EXL3_BOTH int quotient(int n, const Divisor &d) {
  return d.mul == 0u ? n : (int)((uint32_t)(((uint64_t)(uint32_t)n * d.mul) >> 32) >> d.shift);
}

// What the kind settles, so that the compiler knows it (64 sequences over 24000
// shared keys 81.9 -> 80.9 us, 40 of questions 46.5 -> 45.7).
template <int KIND>
EXL3_BOTH int causal_of(const AttnParams &p) {
  return KIND == ATTN_PREFIX ? 0 : KIND == ATTN_OWN ? 1 : p.causal;
}
template <int KIND>
EXL3_BOTH int window_of(const AttnParams &p) {
  return KIND == ATTN_PREFIX || KIND == ATTN_OWN ? 0 : p.window;
}

// One workgroup's work: rows [tile * R, ...) of a sequence's q_len * group
// rows on one key/value head, and its part of their keys.  Row r is head
// r % group of new token r / group: the heads that share keys and values are
// one tile's rows.
struct Work {
  int seq, tile;
  int split, splits;  // this part of the tile's keys, of how many
  int part_keys;      // keys of a part (splits > 1)
  int q0, q_len;      // the sequence's first query row and their number
  int kv_len;
  int part;           // splits > 1: the part's number among those of all split tiles
  int first;          // ATTN_OWN: the first key
  int item;           // ATTN_PREFIX: the item's number
};

// A sequence's keys by its length in device memory, which nothing has checked.
// Near 2^31 a window's first key, and the steps and look-ups ahead of it, would
// pass 2^31, and a page be looked up before the table.  MAX_LENGTH leaves room for
// where a part of a window and first tokens can start: up to 2^20 places past the
// window, and 127 for each of 4096 parts.
EXL3_BOTH int counted_keys(int kv_len) { return least(most(0, kv_len), MAX_LENGTH); }

// The keys that a workgroup reads, [lo, hi), of those the tile's rows r0 ..
// r_last see, and the multiple of 32 where it starts.
struct KeyRange {
  int shift;            // a new token's position is its index + shift
  int p_first, p_last;  // positions of the first and the last row
  int start, lo, hi;
  int end;              // where the workgroup's steps end: hi, but see sink_range
  int sinks, sink_end, skip;
};

template <int KIND = ATTN_PLAIN>
EXL3_BOTH KeyRange key_range(const AttnParams &p, const Work &w, int r0, int r_last) {
  KeyRange k;
  k.shift = w.kv_len - w.q_len;
  k.p_first = k.shift + quotient(r0, p.by_group);
  k.p_last = k.shift + quotient(r_last, p.by_group);
  k.hi = causal_of<KIND>(p) ? least(w.kv_len, k.p_last + 1) : w.kv_len;
  if (p.kv_len) k.hi = least(k.hi, p.table_keys);  // past the table everything is a hole
  k.lo = window_of<KIND>(p) > 0 ? most(0, k.p_first - window_of<KIND>(p) + 1) : 0;
  if constexpr (KIND == ATTN_OWN) k.lo = w.first;
  if (w.splits > 1) {
    const int64_t from = (int64_t)(k.lo & ~31) + (int64_t)w.split * w.part_keys;
    k.lo = (int)least<int64_t>(most<int64_t>(from, k.lo), MAX_KEYS);
    k.hi = (int)least<int64_t>(from + w.part_keys, k.hi);
  }
  k.start = k.lo & ~31;
  k.end = k.hi;
  return k;
}

// The same for rows that see a window, lo .. of the first row to hi, and the
// first `sinks` keys.  Steps of whole tiles of G keys go over places: the first
// keys' tiles, then from the multiple of 32 at or below lo on; place x from
// sink_end on is key x + skip.  (Where those tiles reach the window, every place
// is its key.)  Parts are ranges of places; lo and hi stay those of the tile.
template <int G>
EXL3_BOTH KeyRange sink_range(const AttnParams &p, const Work &w, int r0, int r_last) {
  KeyRange k;
  k.shift = w.kv_len - w.q_len;
  k.p_first = k.shift + quotient(r0, p.by_group);
  k.p_last = k.shift + quotient(r_last, p.by_group);
  k.hi = least(w.kv_len, k.p_last + 1);
  if (p.kv_len) k.hi = least(k.hi, p.table_keys);
  k.lo = most(0, k.p_first - p.window + 1);
  k.sinks = least(p.sinks, k.hi);
  k.sink_end = (most(k.sinks, 0) + G - 1) & ~(G - 1);
  k.skip = most(0, (k.lo & ~31) - k.sink_end);
  k.end = most(k.hi - k.skip, least(k.hi, k.sink_end));  // (the table may end before the window)
  k.start = 0;
  if (w.splits > 1) {
    const int64_t from = (int64_t)w.split * w.part_keys;
    k.start = (int)least<int64_t>(from, MAX_KEYS);
    k.end = (int)least<int64_t>(from + w.part_keys, k.end);
  }
  return k;
}

}  // namespace exl3
