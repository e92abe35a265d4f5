// The keys that the attention kernels' steps reach, for lengths up to the type's
// ends: every key that a step, or a look-up of pages up to three steps ahead,
// computes fits 32 bits and is none below zero, so that the comparisons with the
// range's end and the table's width keep the look-up inside the table.
#include <cstdio>
#include <cstring>

#include "../../linear_exl3_input_amd/csrc/attn_ranges.hpp"

using namespace exl3;

static long g_checked = 0, g_bad = 0;

// Steps go from `start` to `end` in 32s or in tiles of up to 128 keys; places
// from sink_end on are `skip` keys further.
static void check(const KeyRange &k, int sink_end, int skip, const char *what, const AttnParams &p, const Work &w) {
  auto place = [&](int64_t x) {
    const int64_t key = (x >= sink_end ? x + skip : x) + 31;
    ++g_checked;
    if (key >= 31 && key <= 0x7FFFFFFF) return;
    if (g_bad++ < 20)
      std::printf("%s: kv_len %d, %d rows, window %d, sinks %d, table of %d keys, part %d of %d: place %lld is key %lld\n", what,
                  w.kv_len, w.q_len, p.window, p.sinks, p.table_keys, w.split, w.splits, (long long)x, (long long)key);
  };
  constexpr int AHEAD = 96 + 3 * 128 + 96;
  for (int x = 0; x <= AHEAD; x += 32) {
    place((int64_t)k.start + x);
    if (k.end > k.start) place((int64_t)k.end - 1 + x);
  }
}

template <int G>
static void sinks(const AttnParams &p, const Work &w, int r0, int r_last) {
  const KeyRange k = sink_range<G>(p, w, r0, r_last);
  check(k, k.sink_end, k.skip, "first tokens", p, w);
}

int main() {
  const int kvs[] = {(int)0x80000000, -5, 0, 1, 100, 5000, 1 << 20, 1 << 30, MAX_LENGTH - 1, MAX_LENGTH, MAX_LENGTH + 1, MAX_KEYS, 0x7FFFFF00, 0x7FFFFFFE, 0x7FFFFFFF};
  const int rows[] = {1, 2, 90, 1 << 20};
  const int windows[] = {0, 1, 100, 4096, 1 << 29, 1 << 30};
  const int firsts[] = {0, 1, 4, 130, 1 << 20};
  const int64_t tables[] = {0, 16, 4480, 1 << 20, 1 << 30, (1ll << 30) + 4096, 0x7FFFFC00};
  const int of[] = {1, 2, 3, 100, 4096};
  AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.kv_len = kvs;
  p.causal = 1;
  for (int group : {1, 8})
    for (int64_t table : tables)
      for (int window : windows)
        for (int kv : kvs)
          for (int n : rows)
            for (int splits : of) {
              p.group = group;
              p.by_group = Divisor::of((uint32_t)group);
              p.table_keys = (int)least<int64_t>(table, MAX_KEYS);
              p.window = window;
              Work w;
              std::memset(&w, 0, sizeof w);
              w.kv_len = counted_keys(kv);
              w.q_len = n;
              w.splits = splits;
              for (int R : {16, 32, 128}) {
                const int64_t all = (int64_t)n * group;
                for (int64_t r0 : {(int64_t)0, (all - 1) / R * R}) {
                  const int first = (int)r0, last = (int)least<int64_t>(r0 + R, all) - 1;
                  auto parts = [&](int64_t most_seen, auto run) {
                    const int64_t span = least<int64_t>(least(w.kv_len, p.table_keys), most_seen);
                    w.part_keys = (int)(((span + splits - 1) / splits + 127) & ~127);
                    for (int split : {0, 1, splits / 2, splits - 1})
                      if (split < splits) w.split = split, run();
                  };
                  p.sinks = p.sink_keys = 0;
                  parts(window > 0 ? window + R + 32 : 0x7FFFFFFF, [&] {
                    const KeyRange k = key_range<ATTN_PLAIN>(p, w, first, last);
                    check(k, 0x7FFFFFFF, 0, "window", p, w);
                  });
                  if (window == 0) continue;
                  for (int s : firsts) {
                    p.sinks = s;
                    p.sink_keys = (s + 127) & ~127;
                    parts((int64_t)window + R + 32 + p.sink_keys, [&] {
                      sinks<32>(p, w, first, last);
                      sinks<64>(p, w, first, last);
                      sinks<128>(p, w, first, last);
                    });
                  }
                }
              }
            }
  std::printf("places checked: %ld, %ld bad\n", g_checked, g_bad);
  return g_bad != 0;
}
