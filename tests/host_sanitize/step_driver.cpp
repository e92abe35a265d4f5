// Drives the host code of include/exl3_step.h over many sizes and bad
// arguments, built with AddressSanitizer and UndefinedBehaviorSanitizer.
// Device pointers are fake aligned addresses that are never dereferenced.  With
// arguments (batch tokens groups q_heads kv_heads head_dim bits page_width) it
// says which passes a call with shared prefixes makes.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "exl3_step.h"

extern long g_sinks[2], g_shared[2], g_own[2], g_rows, g_tables, g_groups, g_split, g_small, g_tile;
extern uintptr_t g_ws;
extern size_t g_ws_bytes;
static int g_fail = 0;

#define EXPECT(cond)                                                                                                   \
  do {                                                                                                                 \
    if (!(cond)) {                                                                                                     \
      std::fprintf(stderr, "line %d: expected %s (last error: %s)\n", __LINE__, #cond, exl3_last_error());             \
      ++g_fail;                                                                                                        \
    }                                                                                                                  \
  } while (0)

static void *fake(uintptr_t a) { return reinterpret_cast<void *>(a << 40); }
static exl3_rows rows(int heads, int d) { return {fake(1), (int64_t)heads * d, d, heads}; }
static exl3_kv_cache cache(int pages, int page, int heads, int d, int bits) {
  exl3_kv_cache c;
  std::memset(&c, 0, sizeof c);
  c.k = fake(2);
  c.v = fake(3);
  if (bits < 16) c.k_scale = c.v_scale = static_cast<uint8_t *>(fake(4));
  c.k_page_bytes = c.v_page_bytes = (int64_t)heads * page * d * bits / 8;
  if (bits < 16) c.k_scale_page_bytes = c.v_scale_page_bytes = (int64_t)heads * page * d / 32;
  c.pages = pages;
  c.page_size = page;
  c.heads = heads;
  c.head_dim = d;
  c.dtype = EXL3_BF16;
  c.bits = bits;
  return c;
}

static const int32_t *ints = static_cast<const int32_t *>(fake(5));

static exl3_status prefix(int batch, int tokens, int groups, int hq, int hk, int d, int bits, int width, size_t bytes) {
  exl3_kv_cache c = cache(100, 16, hk, d, bits);
  exl3_rows q = rows(hq, d);
  g_ws = reinterpret_cast<uintptr_t>(fake(6));
  g_ws_bytes = bytes;
  return exl3_prefix_attention(&c, &q, &q, ints, ints, ints, width, width, batch, tokens, ints, ints, groups, 0.1f, fake(6),
                               bytes, nullptr);
}

int main(int argc, char **argv) {
  if (argc == 9) {
    int a[8];
    for (int i = 0; i < 8; ++i) a[i] = std::atoi(argv[i + 1]);
    const size_t n = exl3_prefix_attention_workspace_bytes(a[0], a[1], a[2], a[3], a[4], a[5]);
    if (prefix(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], n) != EXL3_OK) return 1;
    std::printf("%s %s %s %s\n", g_shared[0] + g_shared[1] ? "shared" : "plain", g_shared[1] ? "tile" : g_shared[0] ? "small" : "none",
                g_own[1] ? "tile" : g_own[0] ? "small" : "none", g_split ? "split" : "whole");
    return 0;
  }
  const int dims[] = {64, 128, 256};
  const int kvs[] = {1, 2, 7, 8, 64, 1024};
  const int groups_of[] = {1, 3, 4, 8, 16};
  const int batches[] = {1, 2, 24, 64, 300, 5000, 65536};
  const int each[] = {1, 2, 5, 16, 63, 300, 4096};
  for (int d : dims)
    for (int hk : kvs)
      for (int g : groups_of) {
        if (hk * g > 1024) continue;
        for (int b : batches)
          for (int n : each) {
            const int64_t tokens = (int64_t)b * n;
            if (tokens > (1 << 20)) continue;
            exl3_rows q = rows(hk * g, d), k = rows(hk, d);
            const size_t plain = exl3_attention_workspace_bytes(b, (int32_t)tokens, hk * g, hk, d);
            g_ws = reinterpret_cast<uintptr_t>(fake(6));
            g_ws_bytes = plain;
            for (int window : {1, 500, 1 << 30})
              for (int sinks : {0, 4, 1 << 20})
                for (int width : {0, 1, 300, 0x7FFFFFFF}) {
                  exl3_kv_cache c = cache(100, 16, hk, d, n % 2 ? 8 : 16);
                  EXPECT(exl3_paged_attention_sinks(&c, &q, &q, ints, ints, ints, 1ll << 33, width, b, (int32_t)tokens, 0.1f,
                                                    window, sinks, plain ? fake(6) : nullptr, plain, nullptr) == EXL3_OK);
                  if (width == 0)
                    EXPECT(exl3_prompt_attention_sinks(&q, &k, &k, &q, ints, b, (int32_t)tokens, d, EXL3_F16, window, sinks,
                                                       0.1f, plain ? fake(6) : nullptr, plain, nullptr) == EXL3_OK);
                }
            for (int groups : {0, 1, b / 3, b}) {
              const size_t bytes = exl3_prefix_attention_workspace_bytes(b, (int32_t)tokens, groups, hk * g, hk, d);
              EXPECT(exl3_last_error()[0] == 0 && bytes > 0);
              for (int width : {1, 5000, 0x7FFFFFFF}) {
                EXPECT(prefix(b, (int32_t)tokens, groups, hk * g, hk, d, 8, width, bytes) == EXL3_OK);
                EXPECT(prefix(b, (int32_t)tokens, groups, hk * g, hk, d, 8, width, bytes - 1) == EXL3_ERR_WORKSPACE);
              }
            }
          }
      }
  EXPECT(g_sinks[0] && g_sinks[1] && g_shared[0] && g_shared[1] && g_own[0] && g_own[1] && g_groups && g_split && g_small && g_tile);
  exl3_rotary_axes r;
  std::memset(&r, 0, sizeof r);
  r.rotary = {static_cast<float *>(fake(7)), 100, 64, 0};
  r.axes = 3;
  for (int i = 0; i < 8; ++i) r.axis_of[i] = 0x24924924u;
  exl3_head_norm norm = {static_cast<float *>(fake(8)), static_cast<float *>(fake(8)), 32, 1, 1e-6f};
  for (int d : dims)
    for (int bits : {16, 8, 4})
      for (int t : {0, 1, 1000, 1 << 20}) {
        exl3_kv_cache c = cache(64, 256, 8, d, bits);
        exl3_rows q = rows(32, d), k = rows(8, d), out{fake(9), 32 * (int64_t)d, d, 32};
        for (const exl3_head_norm *n : {(const exl3_head_norm *)nullptr, (const exl3_head_norm *)&norm}) {
          EXPECT(exl3_norm_rope(&r, n, ints, 1ll << 40, t, d, EXL3_F16, &q, &out, nullptr, nullptr, nullptr) == EXL3_OK);
          EXPECT(exl3_norm_rope_cache_write(&c, &r, n, ints, t, ints, t, &q, &out, &k, nullptr, &k, nullptr) == EXL3_OK);
        }
      }
  auto at = [](uintptr_t n) { return static_cast<int32_t *>(fake(10 + n)); };
  for (int b : {0, 1, 255, 65536})
    for (int t : {0, 1, 1 << 20})
      for (int width : {0, 1, 0x7FFFFFFF})
        EXPECT(exl3_cache_extend(64, 1024, at(0), at(1), b, at(100000), 1ll << 31, width, at(3), t, t & 1 ? at(4) : nullptr, t, at(5),
                                 at(6), at(7), at(8), at(9), nullptr) == EXL3_OK);
  EXPECT(exl3_cache_extend(64, 1024, at(0), at(1), 65536, at(2), 1ll << 40, 1, at(3), 1, nullptr, 1, at(5), at(6), at(7), at(8),
                           at(2) + (65535ll << 40), nullptr) == EXL3_ERR_INVALID_ARG);
  EXPECT(g_rows > 0 && g_tables > 0);
  std::printf("host checks done: %d failures\n", g_fail);
  return g_fail ? 1 : 0;
}
