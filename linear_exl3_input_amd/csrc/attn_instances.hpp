// Instances of the attention kernels for one head size (EXL3_HEAD_DIM) and
// their launchers; included by one source file per size.
#include "attn_tile.hpp"

namespace exl3 {

namespace {

// Workgroups of a launch: every tile of R rows that `tokens` rows in `batch`
// sequences can make, and the parts that splitting adds (find_work).
int64_t grid_items(const AttnParams &p, int R) {
  return (int64_t)p.tokens * p.group / R + p.batch + p.target;
}

template <bool BF16, int BITS, int NT>
hipError_t small_of(const AttnParams &p, hipStream_t s) {
  const dim3 grid = grid_of(grid_items(p, 16 * NT) * p.heads_kv);
  hipLaunchKernelGGL((attn_small_kernel<BF16, EXL3_HEAD_DIM, BITS, NT>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int NT>
hipError_t small_bits(int bits, const AttnParams &p, hipStream_t s) {
  switch (bits) {
    case 0: return small_of<BF16, 0, NT>(p, s);
    case 4: return small_of<BF16, 4, NT>(p, s);
    case 8: return small_of<BF16, 8, NT>(p, s);
    default: return small_of<BF16, 16, NT>(p, s);
  }
}

template <bool BF16, int BITS>
hipError_t tile_of(const AttnParams &p, hipStream_t s) {
  const dim3 grid = grid_of(grid_items(p, ATTN_TILE_ROWS) * p.heads_kv);
  hipLaunchKernelGGL((attn_tile_kernel<BF16, EXL3_HEAD_DIM, BITS>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

template <bool BF16>
hipError_t tile_bits(int bits, const AttnParams &p, hipStream_t s) {
  switch (bits) {
    case 0: return tile_of<BF16, 0>(p, s);
    case 4: return tile_of<BF16, 4>(p, s);
    case 8: return tile_of<BF16, 8>(p, s);
    default: return tile_of<BF16, 16>(p, s);
  }
}

}  // namespace

#define EXL3_JOIN2(a, b) a##b
#define EXL3_JOIN(a, b) EXL3_JOIN2(a, b)
hipError_t EXL3_JOIN(launch_attn_small_d, EXL3_HEAD_DIM)(bool bf16, int bits, const AttnParams &p, int columns,
                                                         hipStream_t s) {
#if EXL3_HEAD_DIM < 256  // two column tiles of 256-value heads do not fit the registers
  if (columns == 2) return bf16 ? small_bits<true, 2>(bits, p, s) : small_bits<false, 2>(bits, p, s);
#endif
  if (columns != 1) return hipErrorInvalidValue;
  return bf16 ? small_bits<true, 1>(bits, p, s) : small_bits<false, 1>(bits, p, s);
}

hipError_t EXL3_JOIN(launch_attn_tile_d, EXL3_HEAD_DIM)(bool bf16, int bits, const AttnParams &p, hipStream_t s) {
  return bf16 ? tile_bits<true>(bits, p, s) : tile_bits<false>(bits, p, s);
}

}  // namespace exl3
