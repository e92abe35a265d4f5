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

// Probabilities are held as exp2(score - m + LIFT).  The running maximum m
// moves, and what is summed is scaled, only when some row's grew by more than
// LAG, so the largest of a row is between 2^LIFT and 2^(LIFT + LAG).  They are
// rounded to the type for the second product (relative 2^-8 or 2^-11; the sums
// take them unrounded).
// fp16 loses bits below 2^-14 and everything below 2^-25; with LIFT 7 that is
// 2^-21 and 2^-32 of the row's largest, as low as the type's range (2^15 at most)
// lets it be.  With 0, 120000 keys of 1.5 * 2^-24 each beside one of 1 weighed
// 1.42% instead of 1.06%.
// bf16 has fp32's range, and so have its values: what a wave or a part sums
// before it is joined with the others must not be infinite where the result is
// not.  With LIFT -24 the largest is 2^-16 at most, so 65536 keys of the largest
// value fit; what is lost is scores 102 powers of two below the row's largest.
constexpr float PROB_LAG = 8.f;
template <bool BF16>
constexpr float PROB_LIFT = BF16 ? -24.f : 7.f;

// What is subtracted from a row's scores, given its running maximum (-inf: no key yet).
template <bool BF16>
__device__ __forceinline__ float prob_base(float m) {
  return m == -INFINITY ? 0.f : m - PROB_LIFT<BF16>;
}

// The workgroup's number in a grid of grid_of.
__device__ __forceinline__ uint32_t workgroup() { return blockIdx.y << GRID_X_LOG2 | blockIdx.x; }

__device__ __forceinline__ int quotient(int n, const Divisor &d) {
  return d.mul == 0u ? n : (int)(__umulhi((uint32_t)n, d.mul) >> d.shift);
}

// ------------------------------------------------------- codes and scales

// The scale of byte s as a float: 2^(s - 127).  255, a block that held a NaN
// or an infinity, becomes a NaN, and the conversions give NaN for it.  (They
// take the exponent alone, so the zero made of 0 counts as 2^-127.)
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

// Inclusive sums over the wave's lanes by DPP moves: within rows of 16 lanes,
// then row 0's total to row 1, 2's to 3, and the first half's to the second.
__device__ __forceinline__ int wave_inclusive_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return v;
}
// Inclusive maxima of values that are not negative, likewise.
__device__ __forceinline__ int wave_inclusive_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));
  return v;
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_inclusive_sum(v), 63); }
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [&](int moved) __attribute__((always_inline)) { v += __builtin_bit_cast(float, moved); };
  auto bits = [&]() __attribute__((always_inline)) { return __builtin_bit_cast(int, v); };
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x111, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x112, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x114, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x118, 0xF, 0xF, true));
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x142, 0xA, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x143, 0xC, 0xF, false));
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(bits(), 63));
}

// One workgroup's work: rows [tile * R, ...) of a sequence's q_len * group
// rows on one key/value head, and its part of their keys.  Row r is head
// r % group of new token r / group: the heads that share keys and values are
// one tile's rows.
struct Work {
  int seq, tile;
  int split, splits;  // this part of the tile's keys, of how many
  int part_keys;      // keys of a part (splits > 1)
  int q0, q_len;      // the sequence's first query row and their number
  int kv_len;
  int part;           // splits > 1: the part's number among those of all split tiles
};

// Every wave of the workgroup finds the same answer.  Sequence s has
// tiles(s) = ceil(q_len * group / R) tiles.  When the call splits keys, those
// of a sequence whose span (the keys that a tile's rows see at most) exceeds C
// are split into ceil(span / C) equal parts.  C starts as the keys of all
// tiles over `target` and grows twice by what the work items then are over
// `target`, so that they end up near it (whole rounds of the GPU) but for
// lengths that rounding up hits hard; it is at least part_min.  There are
// never more than tiles + target items, nor 2 * target parts.
template <int R>
__device__ __forceinline__ bool find_work(const AttnParams &p, int item, int lane, Work &w) {
  struct Seq {
    int q0, ql, kv, tiles, span;
  };
  // Sequences s0 + lane; `from` is where s0 starts at the earliest, then where
  // the 64 after them do.  An offset below an earlier one counts as that one:
  // sequences never overlap, so what was said above holds whatever cu has.
  auto load = [&](int s0, int &from) __attribute__((always_inline)) -> Seq {
    const int s = s0 + lane;
    int a = 0, b = 0, kv = 0;
    if (s < p.batch) {
      a = p.cu[s], b = p.cu[s + 1];
      if (p.kv_len) kv = p.kv_len[s];
    }
    a = max(from, wave_inclusive_max(min(max(a, 0), p.tokens)));
    b = max(a, min(b, p.tokens));
    from = __builtin_amdgcn_readlane(b, 63);
    Seq x;
    x.q0 = a;
    x.ql = b - a;
    x.kv = p.kv_len ? max(0, kv) : x.ql;
    x.tiles = (int)(((int64_t)x.ql * p.group + R - 1) / R);
    // a tile's rows are at most R tokens; its keys start at a multiple of 32
    x.span = p.kv_len ? min(x.kv, p.table_keys) : x.kv;
    if (p.window > 0) x.span = min(x.span, p.window + R + 32);
    return x;
  };
  int head_end = 0, from;
  const Seq head = load(0, head_end);  // the first 64 sequences, mostly all of them
  auto seq_at = [&](int s0) __attribute__((always_inline)) {
    if (s0 > 0) return load(s0, from);
    from = head_end;
    return head;
  };
  int C = 0x7FFFFFFF;
  auto splits_of = [&](const Seq &x) __attribute__((always_inline)) -> int {
    return x.span > C ? (int)(((uint32_t)x.span + (uint32_t)C - 1u) / (uint32_t)C) : 1;
  };
  if (p.target > 0) {
    // in floats, whose rounding the last factor more than covers: C is never
    // less than keys / target
    float keys = 0.f;
    for (int s0 = 0; s0 < p.batch; s0 += 64) {
      const Seq x = seq_at(s0);
      keys += wave_sum((float)x.tiles * (float)x.span);
    }
    float c = __builtin_fmaxf(keys / (float)p.target * 1.0001f + 1.f, (float)p.part_min);
    for (int i = 0; i < 2; ++i) {
      C = (int)__builtin_fminf(c, 2147483520.f);
      int items = 0;
      for (int s0 = 0; s0 < p.batch; s0 += 64) {
        const Seq x = seq_at(s0);
        items += wave_sum(x.tiles * splits_of(x));
      }
      if (items <= p.target) break;
      c = c * ((float)items / (float)p.target) + 1.f;
    }
    C = (int)__builtin_fminf(c, 2147483520.f);
  }
  int base = 0, pbase = 0;
  for (int s0 = 0; s0 < p.batch; s0 += 64) {
    const Seq x = seq_at(s0);
    const int splits = splits_of(x);
    const int n = x.tiles * splits, parts = splits > 1 ? n : 0;
    const int incl = wave_inclusive_sum(n), pincl = wave_inclusive_sum(parts);
    const uint64_t past = __ballot(item < base + incl);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      w.seq = s0 + l;
      w.splits = __builtin_amdgcn_readlane(splits, l);
      const int at = item - base - __builtin_amdgcn_readlane(incl - n, l);
      w.tile = at / w.splits;
      w.split = at - w.tile * w.splits;
      w.part_keys = ((__builtin_amdgcn_readlane(x.span, l) + w.splits - 1) / w.splits + 127) & ~127;
      w.q0 = __builtin_amdgcn_readlane(x.q0, l);
      w.q_len = __builtin_amdgcn_readlane(x.ql, l);
      w.kv_len = __builtin_amdgcn_readlane(x.kv, l);
      w.part = w.splits > 1 ? pbase + __builtin_amdgcn_readlane(pincl - parts, l) + at : 0;
      // (lengths that are written while the call runs could make more parts than there is room for)
      return w.splits == 1 || w.part - w.split + w.splits <= p.part_cap;
    }
    base += __builtin_amdgcn_readlane(incl, 63);
    pbase += __builtin_amdgcn_readlane(pincl, 63);
  }
  return false;
}

// The keys that a workgroup reads, [lo, hi), of those the tile's rows r0 ..
// r_last see, and the multiple of 32 where it starts.
struct KeyRange {
  int shift;            // a new token's position is its index + shift
  int p_first, p_last;  // positions of the first and the last row
  int start, lo, hi;
};

__device__ __forceinline__ KeyRange key_range(const AttnParams &p, const Work &w, int r0, int r_last) {
  KeyRange k;
  k.shift = w.kv_len - w.q_len;
  k.p_first = k.shift + quotient(r0, p.by_group);
  k.p_last = k.shift + quotient(r_last, p.by_group);
  k.hi = p.causal ? min(w.kv_len, k.p_last + 1) : w.kv_len;
  if (p.kv_len) k.hi = min(k.hi, p.table_keys);  // past the table everything is a hole
  k.lo = p.window > 0 ? max(0, k.p_first - p.window + 1) : 0;
  if (w.splits > 1) {
    const int64_t from = (int64_t)(k.lo & ~31) + (int64_t)w.split * w.part_keys;
    k.lo = (int)min<int64_t>(max<int64_t>(from, k.lo), MAX_KEYS);
    k.hi = (int)min<int64_t>(from + w.part_keys, k.hi);
  }
  k.start = k.lo & ~31;
  return k;
}

// ------------------------------------------------- parts of a split tile
//
// The parts of a tile are added up in a tree of two levels, so that no
// workgroup reads more than a few of them after another: the last of eight
// neighbouring parts' workgroups to arrive adds those eight, in their order,
// and the last of the eights' adds the sums.  Which workgroup does it depends
// on timing, the order of the sum does not.  Parts are written and read with
// device-scope accesses (the workgroups may be on different XCDs); counters
// are zero before and after a call.
constexpr int PART_FAN = 8;
constexpr int ATTN_CPOL_SC1 = 16;  // device-scope coherent access

// The workgroup's stores are made; true in the last of `arrivals` workgroups.
__device__ __forceinline__ bool arrive_last_of(uint32_t *counter, int arrivals) {
  __shared__ int s_last;
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt 0: the wave's stores have been made
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint32_t n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_last = n == (uint32_t)arrivals - 1u;
    if (s_last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return s_last != 0;
}

// After the workgroup has written its part: true in the one workgroup that
// then holds the tile's sum.  add(x0, n, step): the sum of the n parts x0,
// x0 + step, ...; put(x): writes the sum as part x.  Each eight's counter is
// its first part's; the tile's is part 1's, which is no eight's first.
template <class Add, class Put>
__device__ __forceinline__ bool add_parts(const AttnParams &p, const Work &w, int head, Add add, Put put) {
  uint32_t *counters = p.counters + (w.part - w.split) * p.heads_kv + head;
  const int x0 = w.split / PART_FAN * PART_FAN;
  const int n = min(PART_FAN, w.splits - x0);
  if (!arrive_last_of(counters + x0 * p.heads_kv, n)) return false;
  add(x0, n, 1);
  if (w.splits <= PART_FAN) return true;
  put(x0);
  const int eights = (w.splits + PART_FAN - 1) / PART_FAN;
  if (!arrive_last_of(counters + p.heads_kv, eights)) return false;
  add(0, eights, PART_FAN);
  return true;
}

}  // namespace exl3
