// Host-only stand-ins for the attention launchers: each checks the launch it
// is given (grids, the workspace's room, the divisors) as the kernels rely on
// it; nothing touches memory.
#include <cstdio>
#include <cstdlib>

#include "../../linear_exl3_input_amd/csrc/attn_launch.hpp"

extern long g_launches;
long g_small = 0, g_tile = 0;
size_t g_ws_end = 0;  // bytes of the workspace that the last call used

namespace {
void need(bool ok, const char *what) {
  if (!ok) {
    std::fprintf(stderr, "attention launch: %s\n", what);
    std::abort();
  }
}
void check_divisor(const exl3::Divisor &d, uint32_t by) {
  const uint32_t top = 0x7FFFFFFFu;
  const uint32_t ns[] = {0, 1, by - 1, by, by + 1, top, top / by * by, top / by * by - 1, 12345678};
  for (uint32_t n : ns) {
    if (n > top) continue;
    const uint32_t q = d.mul == 0 ? n : (uint32_t)(((uint64_t)n * d.mul) >> 32) >> d.shift;
    need(q == n / by, "divisor");
  }
}
void check_attn(const exl3::AttnParams &p, int R, int D) {
  ++g_launches;
  need(p.tokens > 0 && p.batch > 0 && p.group > 0 && p.heads_kv > 0, "sizes");
  check_divisor(p.by_group, (uint32_t)p.group);
  const long items = (long)((int64_t)p.tokens * p.group / R) + p.batch + p.target;
  need(items * p.heads_kv <= 0x7FFFFFFFl, "grid");
  if (p.target > 0) {
    need(p.counters != nullptr && p.part != nullptr, "workspace");
    need((int64_t)p.part_cap * p.heads_kv * 4 <= 65536, "counters");
    need(p.part_cap >= p.target && p.part_min >= 128, "parts");
    g_ws_end = 65536 + (size_t)p.part_cap * p.heads_kv * R * (D + 2) * 4;
  }
}
}  // namespace

namespace exl3 {
#define EXL3_STUB(D)                                                                                               \
  hipError_t launch_attn_small_d##D(bool, int, const AttnParams &p, int columns, hipStream_t) {                    \
    need(columns == 1 || (columns == 2 && D < 256), "columns");                                                    \
    check_attn(p, 16 * columns, D);                                                                                \
    ++g_small;                                                                                                     \
    return hipSuccess;                                                                                             \
  }                                                                                                                \
  hipError_t launch_attn_tile_d##D(bool, int, const AttnParams &p, hipStream_t) {                                  \
    check_attn(p, ATTN_TILE_ROWS, D);                                                                              \
    ++g_tile;                                                                                                      \
    return hipSuccess;                                                                                             \
  }
EXL3_STUB(64)
EXL3_STUB(128)
EXL3_STUB(256)
hipError_t launch_rows(int, bool, int, const RowsParams &p, hipStream_t) {
  need((int64_t)p.tokens * (p.hq + p.hk + p.hv) < (1ll << 31) && p.tokens > 0, "rows");
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_cache_read(int, bool, int, const ReadParams &p, hipStream_t) {
  need(p.n > 0, "read");
  ++g_launches;
  return hipSuccess;
}
}  // namespace exl3
