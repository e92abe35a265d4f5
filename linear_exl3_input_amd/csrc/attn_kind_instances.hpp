// Instances of the attention kernels for one head size (EXL3_HEAD_DIM) of one
// kind other than the plain one (EXL3_KIND), and their launcher (EXL3_LAUNCH);
// included by one source file per size and kind.
#include "attn_tile.hpp"

namespace exl3 {

namespace {

using Params = std::conditional_t<EXL3_KIND == ATTN_PREFIX, PrefixParams, AttnParams>;

// Two column tiles of 256-value heads do not fit the registers, and own keys
// take one (plan_prefix).
constexpr bool TWO_COLUMNS = EXL3_HEAD_DIM < 256 && EXL3_KIND != ATTN_OWN;

// As many workgroups as a plain launch has.
template <bool BF16, int BITS>
hipError_t launch_columns(const Params &p, int columns, hipStream_t s) {
  const int R = columns > 0 ? 16 * columns : ATTN_TILE_ROWS;
  const dim3 grid = grid_of(((int64_t)p.tokens * p.group / R + p.batch + p.target) * p.heads_kv), block(256);
  if (columns == 0)
    hipLaunchKernelGGL((attn_tile_kernel<BF16, EXL3_HEAD_DIM, BITS, EXL3_KIND, Params>), grid, block, 0, s, p);
  else if (columns == 1)
    hipLaunchKernelGGL((attn_small_kernel<BF16, EXL3_HEAD_DIM, BITS, 1, EXL3_KIND, Params>), grid, block, 0, s, p);
  else if constexpr (TWO_COLUMNS) {
    if (columns != 2) return hipErrorInvalidValue;
    hipLaunchKernelGGL((attn_small_kernel<BF16, EXL3_HEAD_DIM, BITS, 2, EXL3_KIND, Params>), grid, block, 0, s, p);
  } else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_bits(int bits, const Params &p, int columns, hipStream_t s) {
  switch (bits) {
#if EXL3_PACKED
    case 0: return launch_columns<BF16, 0>(p, columns, s);
#endif
    case 4: return launch_columns<BF16, 4>(p, columns, s);
    case 8: return launch_columns<BF16, 8>(p, columns, s);
    case 16: return launch_columns<BF16, 16>(p, columns, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t EXL3_LAUNCH(bool bf16, int bits, const Params &p, int columns, hipStream_t s) {
  return bf16 ? launch_bits<true>(bits, p, columns, s) : launch_bits<false>(bits, p, columns, s);
}

}  // namespace exl3
