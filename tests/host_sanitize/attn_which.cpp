// Which kernel a call of the given sizes runs on and whether its keys are
// split: attn_which <prompt 0|1> <batch> <tokens> <query heads> <key/value heads> <head size>
#include <cstdio>
#include <cstdlib>

#include "exl3_attn.h"

extern long g_small, g_tile;
extern size_t g_ws_end;

int main(int argc, char **argv) {
  if (argc != 7) return 2;
  const int prompt = std::atoi(argv[1]), batch = std::atoi(argv[2]), tokens = std::atoi(argv[3]), hq = std::atoi(argv[4]),
            hkv = std::atoi(argv[5]), d = std::atoi(argv[6]);
  void *p = reinterpret_cast<void *>(1ul << 20);
  const int32_t *ints = static_cast<int32_t *>(p);
  const size_t n = exl3_attention_workspace_bytes(batch, tokens, hq, hkv, d);
  exl3_rows q{p, (int64_t)hq * d, d, hq}, k{p, (int64_t)hkv * d, d, hkv};
  exl3_kv_cache c{};
  c.k = c.v = p;
  c.k_page_bytes = c.v_page_bytes = (int64_t)hkv * 64 * d * 2;
  c.pages = 100;
  c.page_size = 64;
  c.heads = hkv;
  c.head_dim = d;
  c.dtype = EXL3_BF16;
  c.bits = 16;
  const exl3_status st = prompt ? exl3_prompt_attention(&q, &k, &k, &q, ints, batch, tokens, d, EXL3_BF16, 1, 0, 1.f, p, n, nullptr)
                                : exl3_paged_attention(&c, &q, &q, ints, ints, ints, 1, 1, batch, tokens, 1.f, 0, p, n, nullptr);
  if (st != EXL3_OK) {
    std::fprintf(stderr, "%s\n", exl3_last_error());
    return 1;
  }
  std::printf("%s %s\n", g_tile ? "tile" : g_small ? "small" : "none", g_ws_end ? "split" : "whole");
  return 0;
}
