// Attention for many query rows per key/value head: prompts and their chunks.
//
// The mathematics is attn_small.hpp's, one pass with a running maximum, with
// the roles of memory and matrix units turned round: a workgroup of four
// waves has 128 query rows (the heads that share a key/value head times some
// tokens), 32 to a wave, and every tile of keys and values that it reads from
// memory serves all of them.  A tile is BN = 8192 / D keys, so keys and values
// are 16 KB each; 128 threads load the keys and 128 the values, each an 8 x 8
// block (8 rows, 16 bytes of each), one tile ahead in registers and one ahead
// in LDS (two buffers, one barrier a tile).  Codes are decoded on the way to
// LDS, once for all rows.
//
//   S^T[key][row] = K q^T       A = 32 keys x 16 dims, B = 16 dims x 32 rows
//   o^T[dim][row] += V^T p^T    A = 32 dims x 16 keys, B = 16 keys x 32 rows
// A lane holds one row's scores and results (its partner 32 lanes on the
// other half of the keys and dims), so the maximum, the sum and the scaling
// of o are the lane's own.  Again the order of inner indexes is free:
//   - row 8q + 4h + i of a 32-key product takes key 16(q/2) + 8h + 4(q%2) + i,
//     so that the scores of lanes of half h are, 8 at a time, the keys of its
//     part of the second product's B operand;
//   - row m of a 32-dim product takes the dim that spreads the transposed
//     stores over the LDS banks (value_dim), which also leaves every lane
//     with runs of 8 consecutive dims to store.
// In LDS both operands lie as the products read them, 16 bytes a lane and
// consecutive lanes side by side.
#pragma once

#include "attn_small.hpp"

namespace exl3 {

typedef float float16_t __attribute__((ext_vector_type(16)));

template <bool BF16>
__device__ __forceinline__ float16_t mfma32(u32x4_t a, u32x4_t b, float16_t c) {
  if constexpr (BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0,
                                                  0, 0);
}

// The larger (the sum) of a lane's value and its partner's, 32 lanes on.
__device__ __forceinline__ float pair_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int D>
struct TileGeom {
  static constexpr int ROWS = ATTN_TILE_ROWS;  // query rows of a workgroup
  static constexpr int BN = 8192 / D;       // keys of a tile
  static constexpr int NS = BN / 32;        // 32-key products
  static constexpr int NC = D / 8;          // 16-byte pieces of a row
  static constexpr int DT = D / 32;         // 32-dim products
  static constexpr int K_PIECE = BN * 16 + 16;  // LDS bytes of one piece of all keys (and a bank's step)
  static constexpr int K_BYTES = NC * K_PIECE;
  static constexpr int V_BYTES = BN * D * 2;
  static constexpr int BUF = K_BYTES + V_BYTES;
};

template <bool BF16, int D, int BITS>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_tile_kernel(AttnParams p) {
  using G = TileGeom<D>;
  constexpr bool PAGED = BITS != 0;
  constexpr int CB = PAGED ? BITS : 16;
  constexpr int R = G::ROWS, BN = G::BN, NS = G::NS, NC = G::NC, DT = G::DT;
  constexpr int PW = CB / 4;  // words of 8 values: 4, 2 or 1
  __shared__ __align__(16) uint8_t lds[2 * G::BUF];
  __shared__ int s_odd;  // some tile that not all rows see whole has infinities or NaN among its values

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: a wave stages keys or values
  const int col = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % p.heads_kv;
  const int item = blockIdx.x / p.heads_kv;
  Work w;
  if (!find_work<R>(p, item, lane, w)) return;
  const int rows = w.q_len * p.group;
  {
    // a sequence's last tiles have the most keys and go first
    const int tiles = (rows + R - 1) / R;
    w.tile = tiles - 1 - w.tile;
  }

  // ---- the tile's rows and their keys
  const int r0 = w.tile * R;
  const int r_last = min(r0 + R, rows) - 1;
  const KeyRange kr = key_range(p, w, r0, r_last);
  const int lo = kr.lo, hi = kr.hi, p_first = kr.p_first, p_last = kr.p_last, shift = kr.shift;
  const int start = kr.start;
  const int n_tiles = hi > lo ? (hi - start + BN - 1) / BN : 0;

  // ---- the lane's row
  const int r = r0 + 32 * wave + col;
  const bool live = r < rows;
  const int tok = (live ? r : r_last) / p.group;
  const int qh = (live ? r : r_last) - tok * p.group;
  const int pos = shift + tok;
  const int first = p.window > 0 ? max(lo, pos - p.window + 1) : lo;
  const int span = max(0, (p.causal ? min(hi, pos + 1) : hi) - first);
  // of the wave's rows: every one sees [w_lo, w_hi), none beyond w_end
  const int wr0 = min(r0 + 32 * wave, r_last), wr1 = min(wr0 + 31, r_last);
  const int wp0 = shift + wr0 / p.group, wp1 = shift + wr1 / p.group;
  const int w_hi = p.causal ? min(hi, wp0 + 1) : hi, w_end = p.causal ? min(hi, wp1 + 1) : hi;
  const int w_lo = p.window > 0 ? max(lo, wp1 - p.window + 1) : lo;
  const int w_from = p.window > 0 ? max(lo, wp0 - p.window + 1) : lo;

  u32x4_t q[D / 16];
  {
    const uint16_t *a = p.q.data + (int64_t)(w.q0 + tok) * p.q.token + (int64_t)(head * p.group + qh) * p.q.head + 8 * h;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) q[s] = *(const u32x4_t *)(a + 16 * s);
  }

  // ---- staging: thread's block of a tile is rows 8a .. 8a+7, piece c
  const bool stage_v = wave >= 2;
  const int st = tid & 127;
  const int c = st % NC, a8 = 8 * (st / NC);
  const int ps_mask = (1 << p.cache.page_shift) - 1;
  const int32_t *table = PAGED ? p.page_table + (int64_t)w.seq * p.table_stride : nullptr;
  auto page_of = [&](int key) __attribute__((always_inline)) -> int {
    const int i = key >> p.cache.page_shift;
    int pg = -1;
    if (key < hi && i < p.table_width) pg = table[i];
    return pg >= 0 && pg < p.cache.pages ? pg : -1;
  };
  if (tid == 0) s_odd = 0;
  bool holes = false;
  if constexpr (PAGED) {
    int any = 0;
    for (int i = (start >> p.cache.page_shift) + tid; ((int64_t)i << p.cache.page_shift) < hi; i += 256)
      any |= page_of(max(i << p.cache.page_shift, start)) < 0;
    holes = __syncthreads_or(any) != 0;
  }
  uint32_t raw[8][PW];
  uint32_t sc[8];
  auto fetch = [&](int t, int pg) __attribute__((always_inline)) {
    const int key = start + t * BN + a8;
    if constexpr (PAGED) {
      const int pi = max(pg, 0);  // a hole reads page 0; its keys are masked and its values zeroed
      const int64_t row = ((int64_t)head << p.cache.page_shift) + (key & ps_mask);
      const uint8_t *a = (stage_v ? p.cache.v + pi * p.cache.v_page : p.cache.k + pi * p.cache.k_page) +
                         row * (D * CB / 8) + c * CB;
#pragma unroll
      for (int i = 0; i < 8; ++i) load_words(raw[i], a + i * (D * CB / 8));
      if constexpr (CB < 16) {
        const uint8_t *s = (stage_v ? p.cache.v_scale + pi * p.cache.vs_page : p.cache.k_scale + pi * p.cache.ks_page) +
                           row * (D / 32) + (c >> 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) sc[i] = s[i * (D / 32)];
      }
    } else {
      // rows past the last key read as zeros
      const int64_t token = stage_v ? p.v.token : p.k.token;
      const uint16_t *a = (stage_v ? p.v.data + head * p.v.head : p.k.data + head * p.k.head) +
                          (int64_t)(w.q0 + start + t * BN) * token;
      const int step = (int)token * 2;  // the host keeps a tile's rows within 2^31 bytes
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t *>(a), (short)0, (min(hi - start - t * BN, BN) - 1) * step + D * 2, 0x00020000);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u32x4_t x = __builtin_amdgcn_raw_buffer_load_b128(rs, a8 * step + c * 16, i * step, 0);
#pragma unroll
        for (int y = 0; y < 4; ++y) raw[i][y] = x[y];
      }
    }
  };
  // whether every row of the workgroup sees every key of tile t
  auto whole_tile = [&](int t) __attribute__((always_inline)) {
    const int k0 = start + t * BN;
    return k0 >= lo && k0 + BN <= hi && (!p.causal || k0 + BN - 1 <= p_first) &&
           (p.window == 0 || k0 > p_last - p.window) && !holes;
  };
  auto put = [&](int t, int pg) __attribute__((always_inline)) {
    uint8_t *buf = lds + (t & 1) * G::BUF;
    u32x4_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = eight<BF16, CB>(raw[i], 0, CB < 16 ? scale_of(sc[i]) : 1.f);
    if (!stage_v) {
      // key 16t + 8h + 4u + i of each 32 to row 16t + 8u + 4h + i
      const int row = (a8 & ~31) | (a8 & 16) | ((a8 & 8) >> 1);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *(u32x4_t *)(buf + c * G::K_PIECE + (row + (i & 3) + 2 * (i & 4)) * 16) = x[i];
    } else {
      if (!whole_tile(t)) {
        // what lies outside the range or in a hole counts as zero, and so do
        // infinities and NaN that some rows must not see (0 * inf would reach
        // them through the product); the rows that do see them get them below
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = (uint32_t)(start + t * BN + a8 + i - lo) < (uint32_t)(hi - lo) && (!PAGED || pg >= 0);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            x[i][y] = in ? x[i][y] : 0u;
            odd = odd || odd_pair<BF16>(x[i][y]);
            x[i][y] = finite_pair<BF16>(x[i][y]);
          }
        }
        if (odd) s_odd = 1;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
        u32x4_t y;
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = __builtin_amdgcn_perm(x[2 * z + 1][j >> 1], x[2 * z][j >> 1], sel);
        *(u32x4_t *)(buf + G::K_BYTES + ((a8 >> 3) * D + j * NC + c) * 16) = y;
      }
    }
  };

  float16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;  // m: in units of log2, as the scores times scale_log2

  if (n_tiles > 0) {
    int pg = PAGED ? page_of(start + a8) : 0;
    fetch(0, pg);
    __syncthreads();
    put(0, pg);
    if (n_tiles > 1) {
      pg = PAGED ? page_of(start + BN + a8) : 0;
      fetch(1, pg);
    }
    __syncthreads();
    for (int t = 0; t < n_tiles; ++t) {
      if (t + 1 < n_tiles) {
        put(t + 1, pg);
        if (t + 2 < n_tiles) {
          pg = PAGED ? page_of(start + (t + 2) * BN + a8) : 0;
          fetch(t + 2, pg);
        }
      }
      const int k0 = start + t * BN;
      const uint8_t *buf = lds + (t & 1) * G::BUF;
      if (k0 < w_end && k0 + BN > w_from) {
        // ---- scores
        float16_t s[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int n = 0; n < NS; ++n) {
            const u32x4_t a = *(const u32x4_t *)(buf + (2 * d + h) * G::K_PIECE + (32 * n + col) * 16);
            s[n] = mfma32<BF16>(a, q[d], s[n]);
          }
        // ---- mask: element 8t + 4u + i of product n is key k0 + 32n + 16t + 8h + 4u + i
        const bool whole = k0 >= w_lo && k0 + BN <= w_hi && !holes;
        auto sees = [&](int n, int i) __attribute__((always_inline)) {
          return (uint32_t)(k0 + 32 * n + 16 * (i >> 3) + 8 * h + (i & 7) - first) < (uint32_t)span;
        };
        auto hole = [&](int n, int t8) __attribute__((always_inline)) {
          return PAGED && holes && page_of(k0 + 32 * n + 16 * t8 + 8 * h) < 0;
        };
        if (!whole) {
#pragma unroll
          for (int n = 0; n < NS; ++n)
#pragma unroll
            for (int t8 = 0; t8 < 2; ++t8) {
              const bool none = hole(n, t8);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const bool ok = sees(n, 8 * t8 + i) & !none;
                s[n][8 * t8 + i] = ok ? s[n][8 * t8 + i] : -INFINITY;
              }
            }
        }
        // ---- the running maximum; o is scaled only when some row's grew by
        // more than 2^8, so probabilities reach at most 2^8 (exact in range for
        // both types, and the sums are fp32)
        float top = s[0][0];
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[n][i]);
        top = pair_max(top) * p.scale_log2;
        if (__any(top > m + 8.f)) {
          const float grown = __builtin_fmaxf(m, top);
          const float keep = grown == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - grown);
          m = grown;
          l *= keep;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] *= keep;
        }
        const float base = m == -INFINITY ? 0.f : m;
        // ---- probabilities
        u32x4_t pr[NS][2];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int t8 = 0; t8 < 2; ++t8) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * t8 + i], p.scale_log2, -base));
              sum[i & 3] += e[i];
            }
            // rounded to the type for the product; the sum takes them unrounded
#pragma unroll
            for (int y = 0; y < 4; ++y) pr[n][t8][y] = Half<BF16>::pack(e[2 * y], e[2 * y + 1]);
          }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // ---- values
        const uint8_t *vb = buf + G::K_BYTES + col * 16;
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int t8 = 0; t8 < 2; ++t8)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
              const u32x4_t a = *(const u32x4_t *)(vb + ((4 * n + 2 * t8 + h) * D + 32 * d) * 16);
              o[d] = mfma32<BF16>(a, pr[n][t8], o[d]);
            }
      }
      __syncthreads();
    }
  }
  l = pair_sum(l);

  // ---- results: element 4q + i of product d is dim value_dim(d, q, i); for
  // each run of 8 dims (piece) a lane has all 8
  // piece_of: the piece of the lane's run x; (prod, elem): where its j-th dim is.
  auto piece_of = [&](int x) __attribute__((always_inline)) { return D == 64 ? 4 * h + x : 8 * (x >> 2) + 4 * h + (x & 3); };
  auto prod = [](int j) __attribute__((always_inline)) { return D == 64 ? j >> 2 : D == 128 ? j >> 1 : j; };
  auto elem = [](int x, int j) __attribute__((always_inline)) {
    return D == 64 ? 4 * (j & 3) + x : D == 128 ? 4 * (2 * (j & 1) + (x >> 2)) + (x & 3) : x;
  };
  if (n_tiles > 0 && s_odd) {
    // rare: once more over the keys of the tiles that not all rows see whole
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      if (whole_tile(t)) continue;
      const int k0 = start + t * BN;
#pragma unroll 1
      for (int key = max(k0, lo); key < min(k0 + BN, hi); ++key) {
        const int pg = PAGED ? page_of(key) : 0;
        if (pg < 0) continue;
        const bool mine = (uint32_t)(key - first) < (uint32_t)span;
        const int64_t row = ((int64_t)head << p.cache.page_shift) + (key & ps_mask);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int piece = piece_of(x);
          uint32_t word[PW];
          float scale = 1.f;
          if constexpr (PAGED) {
            load_words(word, p.cache.v + pg * p.cache.v_page + row * (D * CB / 8) + piece * CB);
            if constexpr (CB < 16) scale = scale_of(p.cache.v_scale[pg * p.cache.vs_page + row * (D / 32) + (piece >> 2)]);
          } else {
            load_words(word, (const uint8_t *)(p.v.data + (int64_t)(w.q0 + key) * p.v.token + (int64_t)head * p.v.head + 8 * piece));
          }
          const u32x4_t v = eight<BF16, CB>(word, 0, scale);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float f = Half<BF16>::up((v[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
            o[prod(j)][elem(x, j)] += mine && !__builtin_isfinite(f) ? f : 0.f;
          }
        }
      }
    }
  }
  auto store_rows = [&]() __attribute__((always_inline)) {
    if (!live) return;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = o[prod(j)][elem(x, j)];
      store_row<BF16, 8>(p, w, r, head, 8 * piece_of(x), v, l);
    }
  };
  if (w.splits > 1) {
    // a part: [wave][o register / 4][lane][4], then m and the sum of each row
    constexpr int PART = R * (D + 2);
    constexpr int OV = 4 * DT;
    const bool any = r0 + 32 * wave < rows;  // the wave has rows
    auto part_of = [&](int x) __attribute__((always_inline)) {
      return __builtin_amdgcn_make_buffer_rsrc(p.part + ((int64_t)(w.part - w.split + x) * p.heads_kv + head) * PART,
                                               (short)0, PART * 4, 0x00020000);
    };
    auto put = [&](int x) __attribute__((always_inline)) {
      if (!any) return;
      const auto rs = part_of(x);
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int y = 0; y < 4; ++y)
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4_t, (float4_t){o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2], o[d][4 * y + 3]}), rs,
              ((wave * OV + 4 * d + y) * 64 + lane) * 16, 0, ATTN_CPOL_SC1);
      if (h == 0) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(m), rs, (R * D + 32 * wave + col) * 4, 0, ATTN_CPOL_SC1);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(l), rs, (R * D + R + 32 * wave + col) * 4, 0, ATTN_CPOL_SC1);
      }
    };
    auto add = [&](int x0, int count, int step) __attribute__((always_inline)) {
      m = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
      if (!any) return;
      auto row_of = [&](int x, int which) __attribute__((always_inline)) {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(part_of(x0 + x * step), (R * D + which * R + 32 * wave + col) * 4,
                                                                    0, ATTN_CPOL_SC1));
      };
#pragma unroll 4
      for (int x = 0; x < count; ++x) m = __builtin_fmaxf(m, row_of(x, 0));
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
      for (int x = 0; x < count; ++x) {
        const auto rs = part_of(x0 + x * step);
        const float f = __builtin_amdgcn_exp2f(row_of(x, 0) - base);
        l += f * row_of(x, 1);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float4_t v = __builtin_bit_cast(float4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                                rs, ((wave * OV + 4 * d + y) * 64 + lane) * 16, 0, ATTN_CPOL_SC1));
#pragma unroll
            for (int i = 0; i < 4; ++i) o[d][4 * y + i] += v[i] * f;
          }
      }
    };
    put(w.split);
    if (!add_parts(p, w, head, add, put)) return;
  }
  store_rows();
}

}  // namespace exl3
