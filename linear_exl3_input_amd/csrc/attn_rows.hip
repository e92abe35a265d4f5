// Rotary positions and the cache's write and read: kernels that move rows.
#include "attn_rows.hpp"

namespace exl3 {

// ----------------------------------------------- rotation and cache write
//
// A row (one token's one head) is D/8 lanes of one wave, each with 8
// consecutive values.  The rotation pairs a value with its neighbour
// (interleaved) or with the one rot/2 away, which the lane loads too: both
// loads of a row are issued by one wave before any of its stores, so a row
// may be rotated in place.  Quantizing needs the largest magnitude of 32
// values, four neighbouring lanes.
//
// The rows of q, k and v of one token follow one another in the launch, so
// the token's cosines and sines are read from cache for all heads but one.
//
// What bounds it: bytes for prompts, the launch for single steps.  Measured:
// 4099 tokens, 32/8 heads of 128, interleaved, in 15.5 us (86 MB, 5.5 TB/s:
// more than the 4.97 TB/s of a copy, as the output stays in the last cache);
// 16300 tokens written to 8 bits and read back, 8 heads of 128, 46 us for both
// (202 MB, 4.4 TB/s); one step of 16 tokens, 24/4 heads of 256, 3.2 us on the
// GPU and 9.2 with the host's call.
template <bool BF16, int D, int BITS>
__global__ __launch_bounds__(256) void rows_kernel(RowsParams p) {
  constexpr int LPR = D / 8;  // lanes per row
  const int c = threadIdx.x % LPR;
  const int64_t row = (int64_t)workgroup() * (256 / LPR) + threadIdx.x / LPR;
  const int H = p.hq + p.hk + p.hv;
  if (row >= (int64_t)p.tokens * H) return;  // whole rows leave: the quads below stay full
  const uint32_t t = (uint32_t)row / (uint32_t)H;
  int h = (int)((uint32_t)row - t * (uint32_t)H);
  const bool is_q = h < p.hq, is_v = h >= p.hq + p.hk;
  const Rows src = is_q ? p.q : is_v ? p.v : p.k;
  h -= is_q ? 0 : is_v ? p.hq + p.hk : p.hq;
  const uint16_t *x = src.data + (int64_t)t * src.token + (int64_t)h * src.head;
  const u32x4_t own = *(const u32x4_t *)(x + 8 * c);
  uint32_t w[4] = {own.x, own.y, own.z, own.w};
  if (p.table != nullptr && !is_v && 8 * c < p.rot) {
    const int half = p.rot >> 1;
    const int32_t pos = p.positions[t];
    const bool known = pos >= 0 && pos < p.n_positions;
    const float *cs = p.table + (int64_t)(known ? pos : 0) * p.rot;
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Half<BF16>::up(w[i] & 0xFFFFu);
      f[2 * i + 1] = Half<BF16>::up(w[i] >> 16);
    }
    float o[8];
    if (p.interleaved) {
      const float4_t cs0 = *(const float4_t *)(cs + 8 * c), cs1 = *(const float4_t *)(cs + 8 * c + 4);
      const float co[4] = {cs0.x, cs0.z, cs1.x, cs1.z}, si[4] = {cs0.y, cs0.w, cs1.y, cs1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = f[2 * i] * co[i] - f[2 * i + 1] * si[i];
        o[2 * i + 1] = f[2 * i + 1] * co[i] + f[2 * i] * si[i];
      }
    } else {
      const bool second = 8 * c >= half;  // this lane holds the b of its pairs
      const int i0 = second ? 8 * c - half : 8 * c;
      const u32x4_t other = *(const u32x4_t *)(x + (second ? i0 : i0 + half));
      const uint32_t ow[4] = {other.x, other.y, other.z, other.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4_t v = *(const float4_t *)(cs + 2 * i0 + 4 * i);
        const float g0 = Half<BF16>::up(ow[i] & 0xFFFFu), g1 = Half<BF16>::up(ow[i] >> 16);
        const float s0 = second ? v.y : -v.y, s1 = second ? v.w : -v.w;
        o[2 * i] = f[2 * i] * v.x + g0 * s0;  // a*cos - b*sin, or b*cos + a*sin
        o[2 * i + 1] = f[2 * i + 1] * v.z + g1 * s1;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = known ? Half<BF16>::pack(o[2 * i], o[2 * i + 1]) : (BF16 ? 0x7FC07FC0u : 0x7E007E00u);
  }
  const u32x4_t res = {w[0], w[1], w[2], w[3]};
  if (is_q) {
    *(u32x4_t *)(p.q_out.data + (int64_t)t * p.q_out.token + (int64_t)h * p.q_out.head + 8 * c) = res;
    return;
  }
  if (!is_v && p.k_out.data != nullptr)
    *(u32x4_t *)(p.k_out.data + (int64_t)t * p.k_out.token + (int64_t)h * p.k_out.head + 8 * c) = res;
  if constexpr (BITS != 0) {
    const int32_t slot = p.slots[t];
    const int32_t page = slot >> p.cache.page_shift;
    if (slot < 0 || page >= p.cache.pages) return;
    const int off = slot & ((1 << p.cache.page_shift) - 1);
    const int64_t r = ((int64_t)h << p.cache.page_shift) + off;  // the row within its page
    uint8_t *codes = is_v ? p.cache.v + page * p.cache.v_page : p.cache.k + page * p.cache.k_page;
    uint8_t *scales = BITS == 16 ? nullptr : is_v ? p.cache.v_scale + page * p.cache.vs_page
                                                  : p.cache.k_scale + page * p.cache.ks_page;
    write_codes<BF16, D, BITS>(w, codes + r * (D * BITS / 8), BITS == 16 ? nullptr : scales + r * (D / 32), c);
  }
}

// ------------------------------------------------------------ cache read

template <bool BF16, int D, int BITS>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadParams p) {
  constexpr int LPR = D / 8;
  const int c = threadIdx.x % LPR;
  const int64_t row = (int64_t)workgroup() * (256 / LPR) + threadIdx.x / LPR;
  const int H = 2 * p.cache.heads;
  if (row >= (int64_t)p.n * H) return;
  const uint32_t t = (uint32_t)row / (uint32_t)H;
  int h = (int)((uint32_t)row - t * (uint32_t)H);
  const bool is_v = h >= p.cache.heads;
  if (is_v) h -= p.cache.heads;
  const int32_t slot = p.slots[t];
  const int32_t page = slot >> p.cache.page_shift;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (slot >= 0 && page < p.cache.pages) {
    const int off = slot & ((1 << p.cache.page_shift) - 1);
    const int64_t r = ((int64_t)h << p.cache.page_shift) + off;
    const uint8_t *codes =
        (is_v ? p.cache.v + page * p.cache.v_page : p.cache.k + page * p.cache.k_page) + r * (D * BITS / 8);
    if constexpr (BITS == 16) {
      const u32x4_t v = *(const u32x4_t *)(codes + 16 * c);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint8_t *scales =
          (is_v ? p.cache.v_scale + page * p.cache.vs_page : p.cache.k_scale + page * p.cache.ks_page) + r * (D / 32);
      const float s = scale_of(scales[c >> 2]);
      if constexpr (BITS == 8) {
        const u32x2_t v = *(const u32x2_t *)(codes + 8 * c);
        w[0] = Half<BF16>::template fp8<false>(v.x, s);
        w[1] = Half<BF16>::template fp8<true>(v.x, s);
        w[2] = Half<BF16>::template fp8<false>(v.y, s);
        w[3] = Half<BF16>::template fp8<true>(v.y, s);
      } else {
        const uint32_t v = *(const uint32_t *)(codes + 4 * c);
        w[0] = Half<BF16>::template fp4<0>(v, s);
        w[1] = Half<BF16>::template fp4<1>(v, s);
        w[2] = Half<BF16>::template fp4<2>(v, s);
        w[3] = Half<BF16>::template fp4<3>(v, s);
      }
    }
  }
  const Rows dst = is_v ? p.v_out : p.k_out;
  *(u32x4_t *)(dst.data + (int64_t)t * dst.token + (int64_t)h * dst.head + 8 * c) = (u32x4_t){w[0], w[1], w[2], w[3]};
}

// ------------------------------------------------------------- launchers

namespace {

template <bool BF16, int D>
hipError_t rows_of(int bits, const RowsParams &p, hipStream_t s) {
  constexpr int RPB = 256 / (D / 8);
  const int64_t rows = (int64_t)p.tokens * (p.hq + p.hk + p.hv);
  const dim3 grid = grid_of((rows + RPB - 1) / RPB), block(256);
  switch (bits) {
    case 0: hipLaunchKernelGGL((rows_kernel<BF16, D, 0>), grid, block, 0, s, p); break;
    case 4: hipLaunchKernelGGL((rows_kernel<BF16, D, 4>), grid, block, 0, s, p); break;
    case 8: hipLaunchKernelGGL((rows_kernel<BF16, D, 8>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((rows_kernel<BF16, D, 16>), grid, block, 0, s, p); break;
  }
  return hipGetLastError();
}

template <bool BF16, int D>
hipError_t read_of(int bits, const ReadParams &p, hipStream_t s) {
  constexpr int RPB = 256 / (D / 8);
  const int64_t rows = (int64_t)p.n * 2 * p.cache.heads;
  const dim3 grid = grid_of((rows + RPB - 1) / RPB), block(256);
  switch (bits) {
    case 4: hipLaunchKernelGGL((cache_read_kernel<BF16, D, 4>), grid, block, 0, s, p); break;
    case 8: hipLaunchKernelGGL((cache_read_kernel<BF16, D, 8>), grid, block, 0, s, p); break;
    default: hipLaunchKernelGGL((cache_read_kernel<BF16, D, 16>), grid, block, 0, s, p); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(int head_dim, bool bf16, int bits, const RowsParams &p, hipStream_t s) {
  if (bf16)
    return head_dim == 64 ? rows_of<true, 64>(bits, p, s) : head_dim == 128 ? rows_of<true, 128>(bits, p, s)
                                                                            : rows_of<true, 256>(bits, p, s);
  return head_dim == 64 ? rows_of<false, 64>(bits, p, s) : head_dim == 128 ? rows_of<false, 128>(bits, p, s)
                                                                           : rows_of<false, 256>(bits, p, s);
}

hipError_t launch_cache_read(int head_dim, bool bf16, int bits, const ReadParams &p, hipStream_t s) {
  if (bf16)
    return head_dim == 64 ? read_of<true, 64>(bits, p, s) : head_dim == 128 ? read_of<true, 128>(bits, p, s)
                                                                            : read_of<true, 256>(bits, p, s);
  return head_dim == 64 ? read_of<false, 64>(bits, p, s) : head_dim == 128 ? read_of<false, 128>(bits, p, s)
                                                                           : read_of<false, 256>(bits, p, s);
}

}  // namespace exl3
