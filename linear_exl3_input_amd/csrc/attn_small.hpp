// Attention for few query rows per key/value head: one new token a sequence,
// a handful of drafted ones, or any call too small for the large tiles.
//
// With S = scale * q K^T, p = exp2(S * log2(e) - m), o = (p V) / sum(p): one
// pass over the keys with a running maximum m and sum.  A workgroup has 16
// (or 32) query rows, the heads that share a key/value head and a few tokens,
// as the columns of matrix products and a range of keys as the other side:
//   S^T[key][row] = K q^T       A = 16 keys x 32 dims, B = 32 dims x 16 rows
//   o^T[dim][row] += V^T p^T    A = 16 dims x 32 keys, B = 32 keys x 16 rows
// Its four waves take steps of 32 keys in turn, each with its own m, sum and
// o, and add them up at the end; nothing is shared before that, so keys and
// values go from memory to registers without LDS.  The order of a product's
// inner index is free, which settles the rest:
//   - the two 16-key tiles of a step take keys {8a + b} and {8a + 4 + b}
//     (a, b < 4), so that the scores a lane holds are those of 8 consecutive
//     keys, exactly the lane's part of the second product's B operand: the
//     probabilities never change lanes.
//   - the dims of the first product follow the 16 bytes a lane loads of a
//     key's row (8, 16 or 32 values).
//   - a lane loads the same D/16 dims of its 8 values' rows, 16 lanes a whole
//     row; one v_perm_b32 per pair of keys turns them into A operands whose
//     row c is dim (D/16) * c + j for operand j.
//
// What bounds it: the cache's bytes where they are many, else a chain of
// waits (lengths, page numbers, rows, the join of waves and of parts).
// Measured: 64 sequences of up to 16000 keys, 8 bits, 32/8 heads of 128, 957
// MB in 177 us, 5.4 TB/s (a streaming read reaches 5.73 here); 3 sequences of
// up to 120000 keys, 4 bits, 24/4 heads of 256, 293 MB in 76 us, 3.9 TB/s (split
// for one workgroup a CU though two fit, and a 4-bit key costs the same vector
// work for half the bytes; split for two, this takes 12% less, but 24 sequences
// of 8000 keys, which then have twice the parts, 38% more); 24 sequences of up
// to 7 tokens over windows of 4096 keys, 64/8 heads of 64, 131 MB in 41 us, 3.2
// TB/s (two columns of products and exponentials to a load);
// one token over 1100 keys, 4.5 MB in 8.9 us; 32 sequences, one token each, over
// windows of 4096 and 4 first tokens, 8 bits, 245 MB in 53 us, 4.6 TB/s.
#pragma once

#include <type_traits>

#include "attn_device.hpp"

namespace exl3 {

// Values a lane takes from a key's row in one load, and the loads per row
// (four lanes share a row).
template <int D, int BITS>
struct KeyRun {
  static constexpr int FIT = BITS == 4 ? 32 : BITS == 8 ? 16 : 8;  // values in 16 bytes
  static constexpr int LEN = FIT < D / 4 ? FIT : D / 4;
  static constexpr int LOADS = D / (4 * LEN);
  static constexpr int WORDS = LEN * (BITS == 4 ? 4 : BITS == 8 ? 8 : 16) / 32;
};

template <int WORDS>
__device__ __forceinline__ void load_words(uint32_t (&w)[WORDS], const uint8_t *a) {
  if constexpr (WORDS == 1) {
    w[0] = *(const uint32_t *)a;
  } else if constexpr (WORDS == 2) {
    const u32x2_t v = *(const u32x2_t *)a;
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const u32x4_t v = *(const u32x4_t *)(a + 16 * i);
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

// 8 values as four pairs, from 16-bit values or codes; `at` counts 8s.
template <bool BF16, int BITS, int WORDS>
__device__ __forceinline__ u32x4_t eight(const uint32_t (&w)[WORDS], int at, float s) {
  if constexpr (BITS == 4) {
    const uint32_t x = w[at];
    return (u32x4_t){Half<BF16>::template fp4<0>(x, s), Half<BF16>::template fp4<1>(x, s),
                     Half<BF16>::template fp4<2>(x, s), Half<BF16>::template fp4<3>(x, s)};
  } else if constexpr (BITS == 8) {
    const uint32_t x = w[2 * at], y = w[2 * at + 1];
    return (u32x4_t){Half<BF16>::template fp8<false>(x, s), Half<BF16>::template fp8<true>(x, s),
                     Half<BF16>::template fp8<false>(y, s), Half<BF16>::template fp8<true>(y, s)};
  } else {
    return (u32x4_t){w[4 * at], w[4 * at + 1], w[4 * at + 2], w[4 * at + 3]};
  }
}

// Pair x of a row's values.
template <bool BF16, int BITS, int WORDS>
__device__ __forceinline__ uint32_t pair_at(const uint32_t (&w)[WORDS], int x, float s) {
  if constexpr (BITS == 4) {
    const uint32_t v = w[x >> 2];
    switch (x & 3) {
      case 0: return Half<BF16>::template fp4<0>(v, s);
      case 1: return Half<BF16>::template fp4<1>(v, s);
      case 2: return Half<BF16>::template fp4<2>(v, s);
      default: return Half<BF16>::template fp4<3>(v, s);
    }
  } else if constexpr (BITS == 8) {
    return x & 1 ? Half<BF16>::template fp8<true>(w[x >> 1], s) : Half<BF16>::template fp8<false>(w[x >> 1], s);
  } else {
    return w[x];
  }
}

// Whether a pair of 16-bit values has an infinity or NaN.
template <bool BF16>
__device__ __forceinline__ bool odd_pair(uint32_t x) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  return (x & E) == E || ((x >> 16) & E) == E;
}

// A pair of 16-bit values with infinities and NaN replaced by 0.
template <bool BF16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  if ((x & E) == E) x &= 0xFFFF0000u;
  if (((x >> 16) & E) == E) x &= 0xFFFFu;
  return x;
}

// The largest (the sum) of the four lanes that hold a column, 16 lanes apart.
__device__ __forceinline__ float column_max(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// N consecutive dims, from d on, of row r of the tile's sequence.
template <bool BF16, int N>
__device__ __forceinline__ void store_row(const AttnParams &p, const Work &w, int r, int head, int d,
                                          const float (&v)[N], float total) {
  const float inv = total == 0.f ? 0.f : 1.f / total;  // a row that sees no key is zero
  const int i = quotient(r, p.by_group), h = r - i * p.group;
  uint16_t *y = p.out.data + (int64_t)(w.q0 + i) * p.out.token + (int64_t)(head * p.group + h) * p.out.head + d;
  uint32_t x[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; ++j) x[j] = Half<BF16>::pack(v[2 * j] * inv, v[2 * j + 1] * inv);
  if constexpr (N == 4) {
    *(u32x2_t *)y = (u32x2_t){x[0], x[1]};
  } else {
#pragma unroll
    for (int j = 0; j < N / 2; j += 4) *(u32x4_t *)(y + 2 * j) = (u32x4_t){x[j], x[j + 1], x[j + 2], x[j + 3]};
  }
}

template <bool BF16, int D, int BITS, int NT, int KIND = ATTN_PLAIN, class Params = AttnParams>
__global__ __launch_bounds__(256, D * NT >= 256 ? 1 : 2) void attn_small_kernel(Params p) {
  constexpr bool PAGED = BITS != 0, SINKS = KIND == ATTN_SINKS;
  constexpr int CB = PAGED ? BITS : 16;  // bits of a stored value
  constexpr int R = 16 * NT;
  constexpr int DV = D / 16;             // dims of a row that a lane holds of the second product
  constexpr int DP = D / 32;             // as pairs
  using KR = KeyRun<D, CB>;
  constexpr int VW = DV * CB >= 32 ? DV * CB / 32 : 1;  // words of a lane's dims of one value row
  __shared__ __align__(16) float s_o[4][4][64][DV + 1];  // [element i][wave][lane][operand j]
  __shared__ float s_m[4][R], s_l[4][R];
  constexpr bool OWN = KIND == ATTN_OWN;
  __shared__ float4_t s_left[OWN ? R : 1][OWN ? D / 4 : 1], s_sums[OWN ? 256 : 1];  // of the shared keys
  __shared__ float2_t s_left_ml[OWN ? R : 1], s_sums_ml[OWN ? 256 : 1];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int head = workgroup() % p.heads_kv;
  const int item = workgroup() / p.heads_kv;
  Work w;
  __shared__ std::conditional_t<KIND == ATTN_PREFIX, FewGroups, int> s_groups;
  const FewGroups *few = nullptr;
  if constexpr (KIND == ATTN_PREFIX) {
    if (p.groups.batch < FEW_SEQUENCES) {
      few_groups(p.groups, s_groups, workgroup() == 0);
      few = &s_groups;
    }
  }
  if (!find_work<R, KIND>(p, item, lane, w, few)) return;
  if (KIND == ATTN_PREFIX && w.kv_len <= 0) return;  // nothing is shared, nothing reads the state

  // ---- the tile's rows and their keys
  const int rows = w.q_len * p.group;
  const int r0 = w.tile * R;
  const int r_last = min(r0 + R, rows) - 1;
  const KeyRange kr = SINKS ? sink_range<32>(p, w, r0, r_last) : key_range<KIND>(p, w, r0, r_last);
  const int lo = kr.lo, hi = kr.hi, p_first = kr.p_first, p_last = kr.p_last, shift = kr.shift;
  const int end = SINKS ? kr.end : hi;
  // the key at place x of the steps
  auto key_at = [&](int x) __attribute__((always_inline)) { return SINKS && x >= kr.sink_end ? x + kr.skip : x; };
  // whether some row sees key k, holes aside
  auto useful = [&](int k) __attribute__((always_inline)) {
    return (uint32_t)(k - lo) < (uint32_t)(SINKS ? max(0, hi - lo) : hi - lo) || (SINKS && k < kr.sinks);
  };

  // ---- where keys and values lie
  const int ps_mask = (1 << p.cache.page_shift) - 1;
  const int32_t *table = PAGED ? p.page_table + (int64_t)table_row<KIND>(p, w, few) * p.table_stride
                               : nullptr;
  // lane's keys of a step at k0: first product k0 + 8*(c/4) + c%4 and 4 more,
  // second product k0 + 8*g .. + 7; each within one page (pages hold whole 16s)
  auto page_of = [&](int key) __attribute__((always_inline)) -> int {
    const int i = key >> p.cache.page_shift;
    int pg = -1;
    if (key < hi && i < p.table_width) pg = table[i];
    return pg >= 0 && pg < p.cache.pages ? pg : -1;
  };
  // Pages are looked up two steps ahead: loads complete in order, so a step's
  // rows must not wait for a page number issued after the step before's rows.
  int k0 = kr.start + 32 * wave;
  int pk = 0, pv = 0, pk2 = 0, pv2 = 0;  // pages of this step's and the next step's keys and values
  if constexpr (PAGED) {
    pk = page_of(key_at(k0) + 8 * (c >> 2));
    pv = page_of(key_at(k0) + 8 * g);
    pk2 = page_of(key_at(k0 + 128) + 8 * (c >> 2));
    pv2 = page_of(key_at(k0 + 128) + 8 * g);
  }
  int first[NT], span[NT];  // the keys first .. first + span - 1 are those the lane's row (column c of tile n) sees
  int sink[NT];             // and, with SINKS, 0 .. sink - 1
  const uint16_t *q_row[NT];
  bool live[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = r0 + 16 * n + c;
    live[n] = r < rows;
    const int i = quotient(live[n] ? r : r_last, p.by_group);
    const int h = (live[n] ? r : r_last) - i * p.group;
    const int pos = shift + i;
    first[n] = window_of<KIND>(p) > 0 ? max(lo, pos - window_of<KIND>(p) + 1) : lo;
    span[n] = max(0, (causal_of<KIND>(p) ? min(hi, pos + 1) : hi) - first[n]);
    sink[n] = SINKS ? min(kr.sinks, pos + 1) : 0;
    q_row[n] = p.q.data + (int64_t)(w.q0 + i) * p.q.token + (int64_t)(head * p.group + h) * p.q.head;
  }
  // B operands of the first product: dims in the order the key loads have
  u32x4_t q[NT][D / 32];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int t = 0; t < D / 32; ++t) {
      const int u = t / (KR::LEN / 8), e = t % (KR::LEN / 8);
      q[n][t] = *(const u32x4_t *)(q_row[n] + u * 4 * KR::LEN + g * KR::LEN + 8 * e);
    }

  uint32_t kw[2][KR::LOADS][KR::WORDS], vw[8][VW];
  uint32_t ksc[2][2], vsc[8];  // scale bytes: of a key's row, of the lane's block of a value row
  auto load_k = [&](int at, int pg) __attribute__((always_inline)) {
    const int key = key_at(at) + 8 * (c >> 2) + (c & 3);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t *a;
      const uint8_t *sa = nullptr;
      if constexpr (PAGED) {
        const int64_t r = ((int64_t)head << p.cache.page_shift) + ((key + 4 * t) & ps_mask);
        const int pi = max(pg, 0);  // a hole reads page 0 and is masked
        a = p.cache.k + pi * p.cache.k_page + r * (D * CB / 8);
        if constexpr (CB < 16) sa = p.cache.k_scale + pi * p.cache.ks_page + r * (D / 32);
      } else {
        a = (const uint8_t *)(p.k.data + (int64_t)(w.q0 + min(key + 4 * t, hi - 1)) * p.k.token +
                              (int64_t)head * p.k.head);
      }
#pragma unroll
      for (int u = 0; u < KR::LOADS; ++u) load_words(kw[t][u], a + (u * 4 + g) * KR::LEN * CB / 8);
      if constexpr (CB < 16) {
        if constexpr (D == 64) ksc[t][0] = *(const uint16_t *)sa;
        else if constexpr (D == 128) ksc[t][0] = *(const uint32_t *)sa;
        else {
          const u32x2_t v = *(const u32x2_t *)sa;
          ksc[t][0] = v.x, ksc[t][1] = v.y;
        }
      }
    }
  };
  auto load_v = [&](int at, int pg) __attribute__((always_inline)) {
    const int key0 = key_at(at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int key = key0 + 8 * g + i;
      const uint8_t *a;
      if constexpr (PAGED) {
        const int64_t r = ((int64_t)head << p.cache.page_shift) + (key & ps_mask);
        const int pi = max(pg, 0);
        a = p.cache.v + pi * p.cache.v_page + r * (D * CB / 8) + c * (DV * CB / 8);
        if constexpr (CB < 16) vsc[i] = p.cache.v_scale[pi * p.cache.vs_page + r * (D / 32) + (c * DV) / 32];
      } else {
        a = (const uint8_t *)(p.v.data + (int64_t)(w.q0 + min(key, hi - 1)) * p.v.token + (int64_t)head * p.v.head +
                              c * DV);
      }
      if constexpr (DV * CB < 32) vw[i][0] = *(const uint16_t *)a;
      else load_words(vw[i], a);
    }
  };

  // whether every row sees every key of the step at k (holes aside)
  auto whole_step = [&](int k) __attribute__((always_inline)) {
    if (SINKS && k + 32 <= min(kr.sinks, p_first + 1)) return true;
    return k >= lo && k + 32 <= hi && (!causal_of<KIND>(p) || k + 31 <= p_first) && (window_of<KIND>(p) == 0 || k > p_last - window_of<KIND>(p));
  };

  float4_t o[NT][DV];
  float m[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.f;
#pragma unroll
    for (int j = 0; j < DV; ++j) o[n][j] = (float4_t){0.f, 0.f, 0.f, 0.f};
  }

  if (k0 < end) {
    load_k(k0, pk);
    load_v(k0, pv);
  }
  // What the shared keys' parts left for the tile's rows, to LDS: a thread has 4
  // dims of a row and all parts, or, of many, every fourth, whose sums then meet.
  // The first part of the own keys does it, while its first keys are on their
  // way.  64 sequences of up to 1500 own keys, 8 heads of 128, 32 parts: 39 us
  // with the 34 MB that these left, 31 with one part (a lane of the rows alone,
  // after the last key: 49).
  auto collect = [&]() __attribute__((always_inline)) {
    constexpr int Q = D / 4;  // threads of a row
    constexpr int U = 8;      // parts in flight (16: no faster)
    const int n_rows = r_last - r0 + 1;
    const Left all = left_for<D>(p, w, r0, head);
    // loads one after another: either way, a row's parts by one thread or by four
    constexpr int ROWS = 256 / Q;
    const int alone = (n_rows + ROWS - 1) / ROWS * ((all.parts + U - 1) / U);
    const int by_four = (n_rows + ROWS / 4 - 1) / (ROWS / 4) * ((all.parts + 4 * U - 1) / (4 * U));
    const int s_log2 = by_four < alone ? 2 : 0;
    const int q = threadIdx.x % Q, at = threadIdx.x / Q;
    const int part = at & ((1 << s_log2) - 1), rp = at >> s_log2, RP = 256 / Q >> s_log2;
    for (int first_row = 0; first_row < n_rows; first_row += RP) {
      const Left left = left_for<D>(p, w, r0 + min(first_row + rp, n_rows - 1), head);
      float mx = -INFINITY, lx = 0.f;
      float4_t ox = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int x = part; x < left.parts; x += U << s_log2) {
        float2_t ml[U];
        float4_t v[U];
#pragma unroll
        for (int y = 0; y < U; ++y) {
          const float *row = left.row + min(x + (y << s_log2), left.parts - 1) * left.step;
          ml[y] = *(const float2_t *)row;
          v[y] = *(const float4_t *)(row + STATE_PAD + 4 * q);
        }
        float grown = mx;
#pragma unroll
        for (int y = 0; y < U; ++y) grown = __builtin_fmaxf(grown, ml[y].x);
        const float base = grown == -INFINITY ? 0.f : grown;
        const float keep = __builtin_amdgcn_exp2f(mx - base);
        mx = grown;
        lx *= keep;
        ox *= keep;
#pragma unroll
        for (int y = 0; y < U; ++y)
          if (x + (y << s_log2) < left.parts) {
            const float f = __builtin_amdgcn_exp2f(ml[y].x - base);
            lx += ml[y].y * f;
            ox += v[y] * f;
          }
      }
      if (s_log2 > 0) {  // the same for all threads
        __syncthreads();  // the sums of the rows before have been read
        s_sums[threadIdx.x] = ox;
        s_sums_ml[threadIdx.x] = (float2_t){mx, lx};
        __syncthreads();
        if (part == 0) {
#pragma unroll
          for (int y = 1; y < 4; ++y) {
            const float2_t ml = s_sums_ml[threadIdx.x + y * Q];
            const float grown = __builtin_fmaxf(mx, ml.x), base = grown == -INFINITY ? 0.f : grown;
            const float keep = __builtin_amdgcn_exp2f(mx - base), f = __builtin_amdgcn_exp2f(ml.x - base);
            mx = grown;
            lx = lx * keep + ml.y * f;
            ox = ox * keep + s_sums[threadIdx.x + y * Q] * f;
          }
        }
      }
      if (part == 0 && first_row + rp < n_rows) {
        s_left[first_row + rp][q] = ox;
        if (q == 0) s_left_ml[first_row + rp] = (float2_t){mx, lx};
      }
    }
    __syncthreads();
  };
  if constexpr (OWN) {
    if (w.first > 0 && w.split == 0) collect();
  }
  bool odd = false;  // some value that not all rows see is an infinity or NaN
  for (; k0 < end; k0 += 128) {
    const bool more = k0 + 128 < end;
    const int key0 = key_at(k0);
    int pk3 = 0, pv3 = 0;
    if constexpr (PAGED) {
      pk3 = page_of(key_at(k0 + 256) + 8 * (c >> 2));
      pv3 = page_of(key_at(k0 + 256) + 8 * g);
    }
    // ---- scores
    float4_t s[NT][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][t] = (float4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        const int u = d / (KR::LEN / 8), e = d % (KR::LEN / 8);
        float sc = 1.f;
        if constexpr (CB < 16) {
          const int block = u * (4 * KR::LEN / 32) + (g * KR::LEN + 8 * e) / 32;
          const uint32_t word = D == 256 && block >= 4 ? ksc[t][1] : ksc[t][0];
          sc = scale_of((word >> (8 * (block & 3))) & 255u);
        }
        const u32x4_t a = eight<BF16, CB>(kw[t][u], e, sc);
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][t] = Half<BF16>::mfma16(a, q[n][d], s[n][t]);
      }
    }
    if (more) load_k(k0 + 128, pk2);
    // ---- mask: key of score (t, i) is key0 + 8g + 4t + i
    const bool hole = PAGED && pv < 0;
    const bool whole = whole_step(key0) && !__any(hole);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][t][i] *= p.scale_log2;
      if (!whole) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 8 * g + 4 * t + i;
            bool ok = (uint32_t)(key - first[n]) < (hole ? 0u : (uint32_t)span[n]);
            if (SINKS) ok = ok || key < (hole ? 0 : sink[n]);
            s[n][t][i] = ok ? s[n][t][i] : -INFINITY;
          }
      }
    }
    // ---- probabilities
    u32x4_t pr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = s[n][0][0];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, s[n][t][i]);
      top = column_max(top);
      if (__any(top > m[n] + PROB_LAG)) {
        const float grown = __builtin_fmaxf(m[n], top);
        const float keep = grown == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[n] - grown);
        m[n] = grown;
        l[n] *= keep;
#pragma unroll
        for (int j = 0; j < DV; ++j) o[n][j] *= keep;
      }
      const float base = prob_base<BF16>(m[n]);
      float pf[8];
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pf[4 * t + i] = __builtin_amdgcn_exp2f(s[n][t][i] - base);
          sum += pf[4 * t + i];
        }
      l[n] += sum;
      pr[n] = (u32x4_t){Half<BF16>::pack(pf[0], pf[1]), Half<BF16>::pack(pf[2], pf[3]), Half<BF16>::pack(pf[4], pf[5]),
                        Half<BF16>::pack(pf[6], pf[7])};
    }
    // ---- values
    if (!whole) {  // keys outside the range or in a hole: whatever is stored there counts as zero
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (hole || !useful(key0 + 8 * g + i)) {
#pragma unroll
          for (int x = 0; x < VW; ++x) vw[i][x] = 0u;
          if constexpr (CB < 16) vsc[i] = 127u;
        }
    }
    float vs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) vs[i] = CB < 16 ? scale_of(vsc[i]) : 1.f;
    // Infinities and NaN of values that some rows must not see are left out
    // here (0 * inf would reach those rows through the product) and given to
    // the rows that do see them below.
    auto products = [&](auto clean) __attribute__((always_inline)) {
#pragma unroll
      for (int x = 0; x < DP; ++x) {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = pair_at<BF16, CB>(vw[i], x, vs[i]);
          if constexpr (decltype(clean)::value) {
            odd = odd || odd_pair<BF16>(u[i]);
            u[i] = finite_pair<BF16>(u[i]);
          }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u32x4_t a;
#pragma unroll
          for (int y = 0; y < 4; ++y) a[y] = __builtin_amdgcn_perm(u[2 * y + 1], u[2 * y], j ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][2 * x + j] = Half<BF16>::mfma16(a, pr[n], o[n][2 * x + j]);
        }
      }
    };
    if (whole) products(std::false_type{});
    else products(std::true_type{});
    if (more) load_v(k0 + 128, pv2);
    pk = pk2, pv = pv2;
    pk2 = pk3, pv2 = pv3;
  }
  if (__any(odd)) {
    // rare: once more over the wave's steps that not all rows see whole
#pragma unroll 1
    for (int at = kr.start + 32 * wave; at < end; at += 128) {
      const int k = key_at(at);
#pragma unroll 1
      for (int key = SINKS ? k : max(k, lo); key < min(k + 32, hi); ++key) {
        const int pg = PAGED ? page_of(key) : 0;
        if (pg < 0 || (SINKS && !useful(key)) || (whole_step(k) && !__any(PAGED && page_of(k + 8 * g) < 0))) continue;
        const int64_t row = ((int64_t)head << p.cache.page_shift) + (key & ps_mask);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d0 = DV * (4 * g + i);  // element i of operand j is dim d0 + j
          uint32_t word[VW];
          float scale = 1.f;
          const uint8_t *a;
          if constexpr (PAGED) {
            a = p.cache.v + pg * p.cache.v_page + row * (D * CB / 8) + d0 * CB / 8;
            if constexpr (CB < 16) scale = scale_of(p.cache.v_scale[pg * p.cache.vs_page + row * (D / 32) + d0 / 32]);
          } else {
            a = (const uint8_t *)(p.v.data + (int64_t)(w.q0 + key) * p.v.token + (int64_t)head * p.v.head + d0);
          }
          if constexpr (DV * CB < 32) word[0] = *(const uint16_t *)a;
          else load_words(word, a);
#pragma unroll
          for (int x = 0; x < DP; ++x) {
            const uint32_t u = pair_at<BF16, CB>(word, x, scale);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float f = Half<BF16>::up(j ? u >> 16 : u & 0xFFFFu);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                o[n][2 * x + j][i] += ((uint32_t)(key - first[n]) < (uint32_t)span[n] || (SINKS && key < sink[n])) &&
                                              !__builtin_isfinite(f)
                                          ? f
                                          : 0.f;
            }
          }
        }
      }
    }
  }

  // ---- the waves' results together: wave i sums element i of every tile
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] = column_sum(l[n]);
    if (g == 0) {
      s_m[wave][16 * n + c] = m[n];
      s_l[wave][16 * n + c] = l[n];
    }
  }
  __syncthreads();
  float top[NT], total[NT], mine[NT][DV];  // of element `wave` of the lane's operands
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    top[n] = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) top[n] = __builtin_fmaxf(top[n], s_m[x][16 * n + c]);
    // a NaN score leaves top as the others' maximum, and its own sum NaN
    const float base = top[n] == -INFINITY ? 0.f : top[n];
    total[n] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) total[n] += s_l[x][16 * n + c] * __builtin_amdgcn_exp2f(s_m[x][16 * n + c] - base);
    const float keep = __builtin_amdgcn_exp2f(m[n] - base);
    if (n > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < DV; ++j) s_o[i][wave][lane][j] = o[n][j][i] * keep;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < DV; ++j)
      mine[n][j] = (s_o[wave][0][lane][j] + s_o[wave][1][lane][j]) + (s_o[wave][2][lane][j] + s_o[wave][3][lane][j]);
  }
  if constexpr (KIND == ATTN_PREFIX) {
    note_items(p, w, head);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (!live[n]) continue;
      float *y = state_row<D>(p, w.item, head, NT == 2 ? 5 : 4, 16 * n + c);
      if (wave == 0 && g == 0) *(float2_t *)y = (float2_t){top[n], total[n]};
#pragma unroll
      for (int j = 0; j < DV; j += 4)
        *(float4_t *)(y + STATE_PAD + DV * (4 * g + wave) + j) =
            (float4_t){mine[n][j], mine[n][j + 1], mine[n][j + 2], mine[n][j + 3]};
    }
    return;
  }
  if constexpr (KIND == ATTN_OWN) {
    if (w.first > 0 && w.split == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2_t ml = s_left_ml[16 * n + c];
        const float grown = __builtin_fmaxf(top[n], ml.x), base = grown == -INFINITY ? 0.f : grown;
        const float keep = __builtin_amdgcn_exp2f(top[n] - base), f = __builtin_amdgcn_exp2f(ml.x - base);
        top[n] = grown;
        total[n] = total[n] * keep + ml.y * f;
#pragma unroll
        for (int j = 0; j < DV; j += 4) {
          const float4_t v = s_left[16 * n + c][(DV * (4 * g + wave) + j) / 4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[n][j + i] = mine[n][j + i] * keep + v[i] * f;
        }
      }
    }
  }
  if (w.splits > 1) {
    // a part: o as [n][wave][lane][DV], then m and the sum of each row; rows
    // that the tile does not have are neither written nor read
    constexpr int PART = R * (D + 2);
    auto part_of = [&](int x) __attribute__((always_inline)) {
      return __builtin_amdgcn_make_buffer_rsrc(p.part + ((int64_t)(w.part - w.split + x) * p.heads_kv + head) * PART,
                                               (short)0, PART * 4, 0x00020000);
    };
    auto put = [&](int x) __attribute__((always_inline)) {
      const auto r = part_of(x);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (!live[n]) continue;
#pragma unroll
        for (int j = 0; j < DV; j += 4)
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4_t, (float4_t){mine[n][j], mine[n][j + 1], mine[n][j + 2], mine[n][j + 3]}), r,
              (((n * 4 + wave) * 64 + lane) * DV + j) * 4, 0, ATTN_CPOL_SC1);
        if (wave == 0 && g == 0) {
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top[n]), r, (R * D + 16 * n + c) * 4, 0, ATTN_CPOL_SC1);
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(total[n]), r, (R * D + R + 16 * n + c) * 4, 0,
                                                ATTN_CPOL_SC1);
        }
      }
    };
    auto add = [&](int x0, int count, int step) __attribute__((always_inline)) {
      constexpr int U = PART_FAN;  // parts in flight
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        top[n] = -INFINITY;
        total[n] = 0.f;
#pragma unroll
        for (int j = 0; j < DV; ++j) mine[n][j] = 0.f;
        if (!live[n]) continue;
#pragma unroll 1
        for (int x = 0; x < count; x += U) {
          float mx[U], lx[U];
          float4_t ox[U][DV / 4];
          float grown = top[n];
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const auto r = part_of(x0 + min(x + y, count - 1) * step);
            mx[y] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (R * D + 16 * n + c) * 4, 0, ATTN_CPOL_SC1));
            lx[y] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (R * D + R + 16 * n + c) * 4, 0, ATTN_CPOL_SC1));
#pragma unroll
            for (int j = 0; j < DV / 4; ++j)
              ox[y][j] = __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                          r, (((n * 4 + wave) * 64 + lane) * DV + 4 * j) * 4, 0, ATTN_CPOL_SC1));
          }
#pragma unroll
          for (int y = 0; y < U; ++y) grown = __builtin_fmaxf(grown, mx[y]);
          const float base = grown == -INFINITY ? 0.f : grown;
          const float keep = __builtin_amdgcn_exp2f(top[n] - base);
          top[n] = grown;
          total[n] *= keep;
#pragma unroll
          for (int j = 0; j < DV; ++j) mine[n][j] *= keep;
#pragma unroll
          for (int y = 0; y < U; ++y)
            if (x + y < count) {
              const float f = __builtin_amdgcn_exp2f(mx[y] - base);
              total[n] += lx[y] * f;
#pragma unroll
              for (int j = 0; j < DV; ++j) mine[n][j] += ox[y][j / 4][j % 4] * f;
            }
        }
      }
    };
    put(w.split);
    if (!add_parts(p, w, head, add, put)) return;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
    if (live[n]) store_row<BF16, DV>(p, w, r0 + 16 * n + c, head, DV * (4 * g + wave), mine[n], total[n]);
}

}  // namespace exl3
