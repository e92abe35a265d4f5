// Device-side pieces of the attention kernels: the two 16-bit types, the
// cache's codes and scales, and the assignment of work to workgroups.
#pragma once

#include "attn_launch.hpp"
#include "exl3_device.hpp"

namespace exl3 {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float float2_t __attribute__((ext_vector_type(2)));

// The 16-bit type of a call: conversions, products, and the values of codes.
template <bool BF16>
struct Half;

template <>
struct Half<true> {
  static __device__ __forceinline__ float up(uint32_t b) { return bf16_bits_to_f32(b); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){lo, hi}, bf16x2_t));
  }
  static __device__ __forceinline__ float4_t mfma16(u32x4_t a, u32x4_t b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t fp8(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI));
  }
  template <int BYTE>
  static __device__ __forceinline__ uint32_t fp4(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, BYTE));
  }
};

template <>
struct Half<false> {
  static __device__ __forceinline__ float up(uint32_t b) { return f16_bits_to_f32(b); }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((float2_t){lo, hi}, half2_t));
  }
  static __device__ __forceinline__ float4_t mfma16(u32x4_t a, u32x4_t b, float4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                  0, 0);
  }
  template <bool HI>
  static __device__ __forceinline__ uint32_t fp8(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, HI));
  }
  template <int BYTE>
  static __device__ __forceinline__ uint32_t fp4(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, BYTE));
  }
};

// ------------------------------------------------------- codes and scales

// The scale of byte s as a float: 2^(s - 127).  255, a block that held a NaN
// or an infinity, becomes a NaN, and the conversions give NaN for it.
__device__ __forceinline__ float scale_of(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FC00000u : s << 23);
}

// Exponent limits that make every stored value exact in the 16-bit type:
// e4m3 values are multiples of 2^(e-9) up to 448 * 2^e, e2m1 of 2^(e-1) up to
// 6 * 2^e; bf16 is kept to its normal range, fp16 to multiples of 2^-24.
template <bool BF16, int BITS>
struct ScaleRange {
  static constexpr int LO = BITS == 8 ? (BF16 ? -117 : -15) : (BF16 ? -125 : -23);
  static constexpr int HI = BITS == 8 ? (BF16 ? 119 : 7) : (BF16 ? 125 : 13);
};

// The scale byte of a block whose largest magnitude has the fp32 bits amax:
// 448 and 7 are both 1.75 * 2^k (k = 8, 2), so the smallest e with
// amax <= 1.75 * 2^(k+e) comes from amax's own exponent and mantissa.
template <bool BF16, int BITS>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const int e = (int)(amax >> 23) - 127 - (BITS == 8 ? 8 : 2) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(min(max(e, ScaleRange<BF16, BITS>::LO), ScaleRange<BF16, BITS>::HI) + 127);
}

// ----------------------------------------------------------------- work

__device__ __forceinline__ int wave_inclusive_sum(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d, 64);
    if (lane >= d) v += t;
  }
  return v;
}

// One workgroup's work: rows [tile * R, ...) of a sequence's q_len * group
// rows on one key/value head, and its part of their keys.  Row r is head
// r % group of new token r / group: the heads that share keys and values are
// one tile's rows.
struct Work {
  int seq, tile;
  int split, splits;   // this part of the tile's keys, of how many
  int q0, q_len;       // the sequence's first query row and their number
  int kv_len;
  int slot;            // the tile's number over all sequences
};

// Every wave of the workgroup finds the same answer.  Sequence s has
// tiles(s) = ceil(q_len * group / R) tiles and, when the call splits keys,
// ceil(span / C) parts of each, span the keys that a tile's rows see at most
// and C the keys of a part: the keys of all tiles over `target` work items, a
// multiple of 128 (a step of the four waves) and at least part_min.
template <int R>
__device__ __forceinline__ bool find_work(const AttnParams &p, int item, int lane, Work &w, int &C) {
  auto shape = [&](int s, int &q0, int &ql, int &kv, int &tiles) __attribute__((always_inline)) {
    q0 = ql = kv = tiles = 0;
    if (s < p.batch) {
      const int a = min(max(p.cu[s], 0), p.tokens), b = min(max(p.cu[s + 1], 0), p.tokens);
      q0 = a;
      ql = max(0, b - a);
      kv = p.kv_len ? max(0, p.kv_len[s]) : ql;
      tiles = (int)(((int64_t)ql * p.group + R - 1) / R);
    }
  };
  // a tile's rows are at most R tokens; its keys start at a multiple of 32
  auto span = [&](int kv) __attribute__((always_inline)) {
    return p.window > 0 ? min(kv, min(p.window, 0x3FFFFFFF) + R + 32) : kv;
  };
  C = 0x7FFFFF80;
  if (p.target > 0) {
    int64_t keys = 0;
    for (int s0 = 0; s0 < p.batch; s0 += 64) {
      int q0, ql, kv, tiles;
      shape(s0 + lane, q0, ql, kv, tiles);
      keys += (int64_t)tiles * span(kv);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) keys += __shfl_xor(keys, d, 64);
    const int64_t c = ((keys + p.target - 1) / p.target + 127) & ~127ll;
    C = (int)min<int64_t>(max<int64_t>(c, p.part_min), 0x7FFFFF80);
  }
  int base = 0, tbase = 0;
  for (int s0 = 0; s0 < p.batch; s0 += 64) {
    int q0, ql, kv, tiles;
    shape(s0 + lane, q0, ql, kv, tiles);
    const int splits = max(1, (int)(((int64_t)span(kv) + C - 1) / C));
    const int n = tiles * splits;
    const int incl = wave_inclusive_sum(n, lane);
    const int tincl = wave_inclusive_sum(tiles, lane);
    const uint64_t past = __ballot(item < base + incl);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      const int excl = base + __shfl(incl - n, l, 64);
      w.seq = s0 + l;
      w.splits = __shfl(splits, l, 64);
      const int at = item - excl;
      w.tile = at / w.splits;
      w.split = at - w.tile * w.splits;
      w.q0 = __shfl(q0, l, 64);
      w.q_len = __shfl(ql, l, 64);
      w.kv_len = __shfl(kv, l, 64);
      w.slot = tbase + __shfl(tincl - tiles, l, 64) + w.tile;
      return true;
    }
    base += __shfl(incl, 63, 64);
    tbase += __shfl(tincl, 63, 64);
  }
  return false;
}

}  // namespace exl3
