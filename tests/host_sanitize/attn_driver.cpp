// Drives the attention C ABI's host code over many sizes and bad arguments,
// built with AddressSanitizer and UndefinedBehaviorSanitizer.  Device pointers
// are fake aligned addresses that are never dereferenced.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "exl3_attn.h"

extern long g_launches, g_small, g_tile;
extern size_t g_ws_end;
static int g_fail = 0;

#define EXPECT(cond)                                                                               \
  do {                                                                                             \
    if (!(cond)) {                                                                                 \
      std::fprintf(stderr, "line %d: expected %s (last error: %s)\n", __LINE__, #cond, exl3_last_error()); \
      ++g_fail;                                                                                    \
    }                                                                                              \
  } while (0)

static void *fake(uintptr_t a) { return reinterpret_cast<void *>(a << 20); }

static exl3_rows rows(int heads, int d) { return {fake(1), (int64_t)heads * d, d, heads}; }

static exl3_kv_cache cache(int pages, int page, int heads, int d, int bits) {
  exl3_kv_cache c{};
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

int main() {
  const int32_t *ints = static_cast<int32_t *>(fake(5));
  const int dims[] = {64, 128, 256};
  const int kvs[] = {1, 2, 7, 8, 64, 512, 1024};
  const int groups[] = {1, 2, 3, 5, 8, 12, 16};
  const int batches[] = {1, 2, 24, 64, 300, 5000, 65536};
  const int each[] = {1, 2, 5, 16, 63, 300, 4096};
  for (int d : dims)
    for (int hk : kvs)
      for (int g : groups) {
        if (hk * g > 1024) continue;
        for (int b : batches)
          for (int n : each) {
            const int64_t tokens = (int64_t)b * n;
            if (tokens > (1 << 20)) continue;
            const size_t need = exl3_attention_workspace_bytes(b, (int32_t)tokens, hk * g, hk, d);
            EXPECT(exl3_last_error()[0] == 0);
            exl3_rows q = rows(hk * g, d), k = rows(hk, d);
            g_ws_end = 0;
            EXPECT(exl3_prompt_attention(&q, &k, &k, &q, ints, b, (int32_t)tokens, d, EXL3_BF16, 1, 0, 0.1f, need ? fake(6) : nullptr,
                                         need, nullptr) == EXL3_OK);
            EXPECT(g_ws_end <= need);
            exl3_kv_cache c = cache(100, 16, hk, d, n % 2 ? 8 : 16);
            EXPECT(exl3_paged_attention(&c, &q, &q, ints, ints, ints, 1ll << 33, 0x7FFFFFFF, b, (int32_t)tokens, 0.1f, 1 << 30,
                                        need ? fake(6) : nullptr, need, nullptr) == EXL3_OK);
            EXPECT(g_ws_end <= need);
            if (need)
              EXPECT(exl3_paged_attention(&c, &q, &q, ints, ints, ints, 1, 1, b, (int32_t)tokens, 0.1f, 0, fake(6), need - 1,
                                          nullptr) == EXL3_ERR_WORKSPACE);
          }
      }
  EXPECT(g_small > 0 && g_tile > 0);
  exl3_rotary r{static_cast<float *>(fake(7)), 100, 64, 0};
  for (int d : dims)
    for (int bits : {16, 8, 4})
      for (int t : {0, 1, 1000, 1 << 20}) {
        exl3_kv_cache c = cache(64, 256, 8, d, bits);
        exl3_rows q = rows(32, d), k = rows(8, d), out{fake(9), 32 * (int64_t)d, d, 32};
        EXPECT(exl3_rope(&r, ints, t, d, EXL3_F16, &q, &out, nullptr, nullptr, nullptr) == EXL3_OK);
        EXPECT(exl3_cache_write(&c, &k, &k, ints, t, nullptr) == EXL3_OK);
        EXPECT(exl3_rope_cache_write(&c, &r, ints, ints, t, &q, &out, &k, nullptr, &k, nullptr) == EXL3_OK);
        EXPECT(exl3_cache_read(&c, ints, t, &k, &k, nullptr) == EXL3_OK);
      }
  // strides and pages at their limits
  exl3_rows far{fake(1), 1ll << 40, 1ll << 20, 4};
  EXPECT(exl3_rope(&r, ints, 1 << 20, 128, EXL3_BF16, &far, &far, nullptr, nullptr, nullptr) == EXL3_OK);
  far.token_stride = (1ll << 40) + 8;
  EXPECT(exl3_rope(&r, ints, 1, 128, EXL3_BF16, &far, &far, nullptr, nullptr, nullptr) == EXL3_ERR_UNSUPPORTED);
  exl3_kv_cache big = cache(0x7FFFFFFF / 1024, 1024, 1024, 256, 16);
  exl3_rows k = rows(1024, 256);
  EXPECT(exl3_cache_write(&big, &k, &k, ints, 4, nullptr) == EXL3_OK);
  big.pages += 1;
  EXPECT(exl3_cache_write(&big, &k, &k, ints, 4, nullptr) == EXL3_ERR_INVALID_ARG);
  std::printf("host checks done: %d failures, %ld launches\n", g_fail, g_launches);
  return g_fail ? 1 : 0;
}
