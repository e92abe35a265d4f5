// What the kernels that write rows to the cache share.
#pragma once

#include "attn_device.hpp"

namespace exl3 {

// The 8 values of lane c of a row, as pairs, to the row's codes and scales.
// Every lane of the row's quads takes part.
template <bool BF16, int D, int BITS>
__device__ __forceinline__ void write_codes(const uint32_t (&w)[4], uint8_t *codes, uint8_t *scales, int c) {
  if constexpr (BITS == 16) {
    *(u32x4_t *)(codes + 16 * c) = (u32x4_t){w[0], w[1], w[2], w[3]};
  } else {
    float f[8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Half<BF16>::up(w[i] & 0xFFFFu);
      f[2 * i + 1] = Half<BF16>::up(w[i] >> 16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    // the block's four lanes are a DPP quad
    amax = max(amax, __float_as_uint(lane_xor<1>(__uint_as_float(amax))));
    amax = max(amax, __float_as_uint(lane_xor<2>(__uint_as_float(amax))));
    const uint32_t s = scale_byte<BF16, BITS>(amax);
    // 2^-e is exact and normal for every e of ScaleRange; a block that reads
    // as NaN gets zero codes
    const float inv = s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
    constexpr float TOP = BITS == 8 ? 448.f : 6.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = s == 255u ? 0.f : f[i] * inv;
      f[i] = __builtin_fminf(__builtin_fmaxf(y, -TOP), TOP);
    }
    if constexpr (BITS == 8) {
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
      *(u32x2_t *)(codes + 8 * c) = (u32x2_t){(uint32_t)lo, (uint32_t)hi};
    } else {
      uint32_t n = 0;
      n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, f[0], f[1], 1.0f, 0);
      n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, f[2], f[3], 1.0f, 1);
      n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, f[4], f[5], 1.0f, 2);
      n = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(n, f[6], f[7], 1.0f, 3);
      *(uint32_t *)(codes + 4 * c) = n;
    }
    if ((c & 3) == 0) scales[c >> 2] = (uint8_t)s;
  }
}

}  // namespace exl3
