// The attention launches' grids: below 2^32 threads along x, within the other
// dimensions' limit, every workgroup once.
#include <cstdio>

#include "../../linear_exl3_input_amd/csrc/attn_launch.hpp"

int main() {
  int bad = 0;
  const int64_t at[] = {1, 2, 255, 256, 65535, 65536, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, (1 << 24) - 1, 1 << 24,
                        3 << 23, 12345678, 1 << 28, (1 << 28) + 1, 2147483646, 2147483647};
  for (int64_t n : at) {
    const dim3 g = exl3::grid_of(n);
    const int64_t last = (int64_t)(g.y - 1) << exl3::GRID_X_LOG2;  // the last row's first workgroup
    const bool ok = (int64_t)g.x * 256 < (1ll << 32) && g.y >= 1 && g.y <= 65535 && g.z == 1 && last < n && last + g.x >= n &&
                    (g.y == 1 ? g.x == n : g.x == 1u << exl3::GRID_X_LOG2) &&
                    (((int64_t)g.y << exl3::GRID_X_LOG2) <= (1ll << 31) || g.y == 1);
    if (!ok) std::printf("%lld workgroups: %u x %u x %u\n", (long long)n, g.x, g.y, g.z), ++bad;
  }
  std::printf("grids checked: %d bad\n", bad);
  return bad != 0;
}
