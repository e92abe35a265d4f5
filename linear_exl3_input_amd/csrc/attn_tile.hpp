// Attention for many query rows per key/value head: prompts and their chunks.
//
// The mathematics is attn_small.hpp's, one pass with a running maximum, with
// the roles of memory and matrix units turned round: a workgroup of four
// waves has 128 query rows (the heads that share a key/value head times some
// tokens), 32 to a wave, and every tile of keys and values that it reads from
// memory serves all of them.  A tile is BN = 8192 / D keys, so keys and values
// are 16 KB each.  Of every tile a thread stages 4 pieces (8 dims) of keys and
// 8 half pieces of values, which it turns so that keys lie side by side; both
// go through registers, a tile ahead of LDS, into two buffers (one barrier a
// tile).  Codes are decoded on the way, once for all rows.
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
//
// A turn of the loop is two runs of 16 steps: the scores of tile t with the
// staging beside them, then the products with the values of tile t - 1 with
// the exponentials of tile t and the loads of tile t + 2 beside them, so that
// matrix, vector and memory work go on together.  The order is written out
// and held by scheduling barriers; with it, staging by every wave and the
// products' results in VGPRs, windows with heads of 256 went from 403 to 283
// us and prompts of up to 8000 tokens from 1004 to 982.
//
// What bounds it: vector work about as long as the products, on the same
// SIMDs.  A wave-tile is 32 products of 32x32x16 (1024 cycles of its SIMD's
// matrix unit), some 1060 cycles of vector work, half of them exponentials,
// and 32 KB of LDS reads; counters show the matrix units busy for 47% of the
// cycles, the vector units for 52%, the LDS for 37%.  Measured (cards differ by
// up to 10% here): prompts of up to 8000 tokens, 32/8 heads of 128, 931 GFLOP in
// 960-1050 us, 890-970 TFLOP/s (a large matrix product reaches 1283 on the
// fastest); chunks of up to 1000 tokens over up to 20000 keys of 8 bits, 523
// GFLOP in 690-735 us, 710-760; windows of 2048, 24/4 heads of 256, 206 GFLOP in
// 277-295 us, 700-745 (one wave a SIMD, as o alone takes 128 registers); with 16
// first tokens beside windows of 1024, 305 GFLOP in 471 us, 648; chunks of up to 900
// tokens over windows of 2048 and 100 first tokens, heads of 128, 67 GFLOP in 92-97, 700-733.
// Registers are short: two waves a SIMD have 256 each, which heads of 64 and
// 128 fill; over codes and with heads of 64 over 16-bit caches 1 to 14 registers
// are kept in memory, elsewhere none.  64 rows a wave halve the LDS reads but
// do not fit; eight waves as two groups of four that alternate products and
// vector work took 925 us on the first (where this took 960) but more on chunks,
// and do not fit with heads of 256.
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
  static constexpr int BN = 8192 / D;       // keys of a tile
  static constexpr int NS = BN / 32;        // 32-key products
  static constexpr int NC = D / 8;          // 16-byte pieces of a row
  static constexpr int DT = D / 32;         // 32-dim products
  static constexpr int K_PIECE = BN * 16 + 16;  // LDS bytes of one piece of all keys (and a bank's step)
  static constexpr int K_BYTES = NC * K_PIECE;
  static constexpr int V_BYTES = BN * D * 2;
  static constexpr int BUF = K_BYTES + V_BYTES;
};

template <bool BF16, int D, int BITS, int KIND = ATTN_PLAIN, class Params = AttnParams>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_tile_kernel(Params p) {
  using G = TileGeom<D>;
  constexpr bool PAGED = BITS != 0, SINKS = KIND == ATTN_SINKS;
  constexpr int CB = PAGED ? BITS : 16;
  constexpr int R = ATTN_TILE_ROWS, BN = G::BN, NS = G::NS, NC = G::NC, DT = G::DT;
  constexpr int PW = CB / 4;  // words of 8 values: 4, 2 or 1
  __shared__ __align__(16) uint8_t lds[2 * G::BUF];
  __shared__ int s_odd;  // some tile that not all rows see whole has infinities or NaN among its values

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: a wave stages keys or values
  const int col = lane & 31, h = lane >> 5;
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
  const int rows = w.q_len * p.group;
  if constexpr (KIND != ATTN_PREFIX) {
    // a sequence's last tiles have the most keys and go first
    const int tiles = (rows + R - 1) / R;
    w.tile = tiles - 1 - w.tile;
  }

  // ---- the tile's rows and their keys
  const int r0 = w.tile * R;
  const int r_last = min(r0 + R, rows) - 1;
  const KeyRange kr = SINKS ? sink_range<BN>(p, w, r0, r_last) : key_range<KIND>(p, w, r0, r_last);
  const int lo = kr.lo, hi = kr.hi, p_first = kr.p_first, p_last = kr.p_last, shift = kr.shift;
  const int start = kr.start;
  const int n_tiles = SINKS ? max(0, kr.end - start + BN - 1) / BN : hi > lo ? (hi - start + BN - 1) / BN : 0;
  // the first key of tile t
  auto tile_key = [&](int t) __attribute__((always_inline)) {
    const int x = start + t * BN;
    return SINKS && x >= kr.sink_end ? x + kr.skip : x;
  };
  // whether some row sees key k, holes aside
  auto useful = [&](int k) __attribute__((always_inline)) {
    return (uint32_t)(k - lo) < (uint32_t)(SINKS ? max(0, hi - lo) : hi - lo) || (SINKS && k < kr.sinks);
  };

  // ---- the lane's row, which sees the keys first .. first + span - 1
  const int row = r0 + 32 * wave + col;
  const int pos = shift + quotient(min(row, r_last), p.by_group);
  const int first = window_of<KIND>(p) > 0 ? max(lo, pos - window_of<KIND>(p) + 1) : lo;
  const int span = max(0, (causal_of<KIND>(p) ? min(hi, pos + 1) : hi) - first);
  const int sink = SINKS ? min(kr.sinks, pos + 1) : 0;  // and, with SINKS, 0 .. sink - 1
  // of the wave's rows, first to last, every one sees [w_lo, w_hi)
  const int wp0 = shift + quotient(min(r0 + 32 * wave, r_last), p.by_group);
  const int wp1 = shift + quotient(min(r0 + 32 * wave + 31, r_last), p.by_group);
  const int w_hi = causal_of<KIND>(p) ? min(hi, wp0 + 1) : hi, w_lo = window_of<KIND>(p) > 0 ? max(lo, wp1 - window_of<KIND>(p) + 1) : lo;
  const int w_sink = SINKS ? min(kr.sinks, wp0 + 1) : 0;
  // Whole rows pass between memory and the wave's registers through its quarter
  // of LDS (before the first and after the last tile): a row's D / 8 pieces by
  // as many lanes side by side, where the lane's own 16 bytes of 32 rows each
  // would be a line a lane and load (64 prompts of 128 tokens, 32/8 heads of
  // 128: 50 us that way, 44 this; no difference at thousands of tokens).  The
  // pieces of a row are permuted so that neither side meets a bank twice.
  constexpr int RPI = 64 / NC;  // rows of one access
  auto piece_in_lds = [&](int r, int piece) __attribute__((always_inline)) {
    return (u32x4_t *)(lds + wave * (32 * D * 2) + (r * NC + (piece ^ (r & 7))) * 16);
  };
  // Where the tile's row 32 * wave + r is in `x`, as elements (past the last
  // row: the last).
  auto row_offset = [&](const Rows &x, int r) __attribute__((always_inline)) {
    const int at = min(r0 + 32 * wave + r, r_last), t = quotient(at, p.by_group);
    return (int64_t)(w.q0 + t) * x.token + (int64_t)(head * p.group + at - t * p.group) * x.head;
  };
  // The piece of access i that lane `ln` moves, given its own row's offset.
  auto piece_at = [&](const Rows &x, int64_t own, int i, int ln) __attribute__((always_inline)) {
    const int r = i * RPI + ln / NC;
    const uint32_t low = (uint32_t)__shfl((int)own, r, 64), high = (uint32_t)__shfl((int)(own >> 32), r, 64);
    return x.data + (int64_t)((uint64_t)high << 32 | low) + 8 * (ln % NC);
  };
  auto lds_order = [&]() __attribute__((always_inline)) {  // LDS serves a wave's accesses in order
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  };

  // ---- staging: of every tile a thread has piece c (8 dims) of the keys
  // ka .. ka+3 and half of piece c of the values of va .. va+7
  const int c = tid % NC;
  const int ka = 4 * (tid / NC), va = 8 * (tid / (2 * NC));
  const int half = (tid / NC) & 1;
  const int ps_mask = (1 << p.cache.page_shift) - 1;
  const int32_t *table = PAGED ? p.page_table + (int64_t)table_row<KIND>(p, w, few) * p.table_stride
                               : nullptr;
  auto page_of = [&](int key) __attribute__((always_inline)) -> int {
    const int i = key >> p.cache.page_shift;
    int pg = -1;
    if (key < hi && i < p.table_width) pg = table[i];
    return pg >= 0 && pg < p.cache.pages ? pg : -1;
  };
  constexpr int HW = CB == 4 ? 1 : CB / 8;  // words of half a piece (of 4 bits: two bytes)
  constexpr int ROW = D * CB / 8;           // bytes of a cached row
  uint32_t kraw[4][PW], vraw[8][HW];
  uint32_t ksc[4], vsc[8];
  // Packed rows: a descriptor that ends with tile t's last key, so rows past it
  // read as zeros (and nothing is read past the last tile).  The check sees the
  // vector offset alone, so a row's place is there and not in the scalar one.
  auto packed = [&](const Rows &x, int t) __attribute__((always_inline)) {
    const int n = min(hi - tile_key(t), BN);  // the host keeps a tile's rows within 2^31 bytes
    return __builtin_amdgcn_make_buffer_rsrc(x.data + head * x.head + (int64_t)(w.q0 + tile_key(t)) * x.token, (short)0,
                                             n > 0 ? (n - 1) * ((int)x.token * 2) + D * 2 : 0, 0x00020000);
  };
  // The loads of keys tk and values tv, in 12 pieces (4 of keys, 8 of values)
  // for the caller to spread; a page that is none reads page 0, its keys are
  // masked and its values zeroed.
  auto fetch = [&](int tk, int kpg, int tv, int vpg) __attribute__((always_inline)) {
    if constexpr (PAGED) {
      const int64_t kat = ((int64_t)head << p.cache.page_shift) + ((tile_key(tk) + ka) & ps_mask);
      const int64_t vat = ((int64_t)head << p.cache.page_shift) + ((tile_key(tv) + va) & ps_mask);
      const uint8_t *k = p.cache.k + max(kpg, 0) * p.cache.k_page + kat * ROW + c * CB;
      const uint8_t *v = p.cache.v + max(vpg, 0) * p.cache.v_page + vat * ROW + c * CB + half * (CB / 2);
      const uint8_t *ks = nullptr, *vs = nullptr;
      if constexpr (CB < 16) {
        ks = p.cache.k_scale + max(kpg, 0) * p.cache.ks_page + kat * (D / 32) + (c >> 2);
        vs = p.cache.v_scale + max(vpg, 0) * p.cache.vs_page + vat * (D / 32) + (c >> 2);
      }
      return [&, k, v, ks, vs](int i) __attribute__((always_inline)) {
        if (i < 4) {
          load_words(kraw[i], k + i * ROW);
          if constexpr (CB < 16) ksc[i] = ks[i * (D / 32)];
        } else {
          i -= 4;
          if constexpr (CB == 4) vraw[i][0] = *(const uint16_t *)(v + i * ROW);
          else load_words(vraw[i], v + i * ROW);
          if constexpr (CB < 16) vsc[i] = vs[i * (D / 32)];
        }
      };
    } else {
      const auto krs = packed(p.k, tk), vrs = packed(p.v, tv);
      const int kstep = (int)p.k.token * 2, vstep = (int)p.v.token * 2;
      int kat = ka * kstep + c * 16, vat = va * vstep + c * 16 + half * 8;
      asm volatile("" : "+v"(kat), "+v"(vat));  // the rows' offsets made at the loads, not held through the loop
      return [&, krs, vrs, kstep, vstep, kat, vat](int i) __attribute__((always_inline)) {
        if (i < 4) {
          const u32x4_t x = __builtin_bit_cast(
              u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(krs, kat + i * kstep, 0, 0));
#pragma unroll
          for (int y = 0; y < 4; ++y) kraw[i][y] = x[y];
        } else {
          i -= 4;
          const u32x2_t x = __builtin_bit_cast(
              u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(vrs, vat + i * vstep, 0, 0));
          vraw[i][0] = x.x, vraw[i][HW - 1] = x.y;
        }
      };
    }
  };
  // The first loads, and while they are on their way a look at every page for
  // holes and the wait for q (which inside the loop would also be one for the
  // tiles on their way).
  auto key_page = [&](int t, int a) __attribute__((always_inline)) { return PAGED ? page_of(tile_key(t) + a) : 0; };
  int vpg = key_page(0, va);  // of the values in vraw
  int kpg_next = key_page(0, ka), vpg_next = key_page(1, va);
  u32x4_t q[D / 16];
  {
    const int64_t own = row_offset(p.q, col);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) q[i] = *(const u32x4_t *)piece_at(p.q, own, i, lane);
  }
  if (n_tiles > 0) {
    const auto load = fetch(0, kpg_next, 0, vpg);
    kpg_next = key_page(1, ka);
#pragma unroll
    for (int i = 0; i < 12; ++i) load(i);
  }
  if (tid == 0) s_odd = 0;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) *piece_in_lds(i * RPI + lane / NC, lane % NC) = q[i];
  lds_order();
#pragma unroll
  for (int i = 0; i < D / 16; ++i) q[i] = *piece_in_lds(col, 2 * i + h);
  bool holes = false;
  if constexpr (PAGED) {
    int any = 0;
    if constexpr (SINKS) {  // 16 keys, which have one page, at a time: pages that no row sees may be gone
      for (int at = 16 * tid; at < n_tiles * BN; at += 16 * 256) {
        const int x = start + at, k = x >= kr.sink_end ? x + kr.skip : x;
        any |= (k < kr.sinks || (k + 15 >= lo && k < hi)) && page_of(k) < 0;
      }
    } else {
      for (int i = (start >> p.cache.page_shift) + tid; ((int64_t)i << p.cache.page_shift) < hi; i += 256)
        any |= page_of(max(i << p.cache.page_shift, start)) < 0;
    }
    holes = __syncthreads_or(any) != 0;
  } else {
    __syncthreads();
  }
#pragma unroll
  for (int s = 0; s < D / 16; ++s) asm volatile("" : "+v"(q[s]));
  // whether every row of the workgroup sees every key of tile t
  auto whole_tile = [&](int t) __attribute__((always_inline)) {
    const int k0 = tile_key(t);
    if (SINKS && k0 + BN <= min(kr.sinks, p_first + 1)) return !holes;
    return k0 >= lo && k0 + BN <= hi && (!causal_of<KIND>(p) || k0 + BN - 1 <= p_first) &&
           (window_of<KIND>(p) == 0 || k0 > p_last - window_of<KIND>(p)) && !holes;
  };
  // Piece i (0..3) of the thread's keys to tile t's buffer.
  auto put_k = [&](int t, int i) __attribute__((always_inline)) {
    // key 16t + 8h + 4u + i of each 32 to row 16t + 8u + 4h + i
    const int at = (ka & ~12) | ((ka & 8) >> 1) | ((ka & 4) << 1);
    *(u32x4_t *)(lds + (t & 1) * G::BUF + c * G::K_PIECE + (at + i) * 16) =
        eight<BF16, CB>(kraw[i], 0, CB < 16 ? scale_of(ksc[i]) : 1.f);
  };
  // Values of a tile that some row does not see whole: what lies outside the
  // range or in a hole counts as zero, and so do infinities and NaN that some
  // rows must not see (0 * inf would reach them through the product); the rows
  // that do see them get them at the end.  (Those of codes: finite_v.)
  auto clean_v = [&](int t, int pg) __attribute__((always_inline)) {
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool in = useful(tile_key(t) + va + i) && (!PAGED || pg >= 0);
#pragma unroll
      for (int y = 0; y < HW; ++y) {
        vraw[i][y] = in ? vraw[i][y] : 0u;
        if constexpr (CB == 16) {
          odd = odd || odd_pair<BF16>(vraw[i][y]);
          vraw[i][y] = finite_pair<BF16>(vraw[i][y]);
        }
      }
      if constexpr (CB < 16) vsc[i] = in ? vsc[i] : 127u;
    }
    if (odd) s_odd = 1;
  };
  auto values_of = [&](int t) __attribute__((always_inline)) {  // where the thread's values of tile t are
    return lds + (t & 1) * G::BUF + G::K_BYTES + ((va >> 3) * D + 4 * half * NC + c) * 16;
  };
  // Dims 2j and 2j + 1 (j 0..1) of the thread's values, keys side by side.
  auto put_v = [&](int t, int j) __attribute__((always_inline)) {
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = pair_at<BF16, CB>(vraw[i], j, CB < 16 ? scale_of(vsc[i]) : 1.f);
    uint8_t *buf = values_of(t);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      u32x4_t v;
#pragma unroll
      for (int z = 0; z < 4; ++z) v[z] = __builtin_amdgcn_perm(x[2 * z + 1], x[2 * z], y ? 0x07060302u : 0x05040100u);
      *(u32x4_t *)(buf + (2 * j + y) * NC * 16) = v;
    }
  };
  // Codes may stand for infinities and NaN in several ways (a NaN code, a block
  // that held one, a scale that overflows the type), so they are looked for among
  // the decoded values, in LDS, where the thread has put them: on the raw codes
  // this costs registers that the loop does not have (chunks over 8 bits 685 ->
  // 715 us, this way 690; 16-bit values in LDS instead of above: windows with
  // heads of 256 277 -> 294).
  auto finite_v = [&](int t) __attribute__((always_inline)) {
    bool odd = false;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      u32x4_t *at = (u32x4_t *)(values_of(t) + j * NC * 16);
      u32x4_t v = *at;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        odd = odd || odd_pair<BF16>(v[y]);
        v[y] = finite_pair<BF16>(v[y]);
      }
      *at = v;
    }
    if (odd) s_odd = 1;
  };

  float16_t o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;  // m: in units of log2, as the scores times scale_log2
  float16_t s[NS];    // scores
  u32x4_t pr[NS][2];  // probabilities in the type
  constexpr int READS = 16;  // LDS reads of either product of a tile
  constexpr int AHEAD = 3;   // that many are made before their products

  // Tile t's scores, and beside the products the staging of keys t + 1 and
  // values t.  Here and below a step is what is between two scheduling
  // barriers: operands are read AHEAD steps before their products, and the
  // rest is spread so that no step waits for itself or crowds the LDS or the
  // memory path.
  auto score_and_stage = [&](int t) __attribute__((always_inline)) {
    const uint8_t *kb = lds + (t & 1) * G::BUF + h * G::K_PIECE + col * 16;
    auto read = [&](int x) __attribute__((always_inline)) {  // the keys of product x = d * NS + n
      return *(const u32x4_t *)(kb + 2 * (x / NS) * G::K_PIECE + 32 * (x % NS) * 16);
    };
    u32x4_t ring[READS];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[n][i] = 0.f;
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) ring[x] = read(x);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < READS; ++x) {
      if (x + AHEAD < READS) ring[x + AHEAD] = read(x + AHEAD);
      s[x % NS] = mfma32<BF16>(ring[x], q[x / NS], s[x % NS]);
      if (x >= 2 && x < 10 && x % 2 == 0) put_k(t + 1, (x - 2) / 2);
      if (x == 3 || x == 7) put_v(t, x / 4);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The mask, and the running maximum.  True when it moved: o then has to be
  // multiplied by `keep`.
  auto settle = [&](int t, float &keep) __attribute__((always_inline)) -> bool {
    const int k0 = tile_key(t);
    if (!(((k0 >= w_lo && k0 + BN <= w_hi) || (SINKS && k0 + BN <= w_sink)) && !holes)) {
      // element 8t8 + i of product n is key k0 + 32n + 16t8 + 8h + i
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int t8 = 0; t8 < 2; ++t8) {
          const int key = k0 + 32 * n + 16 * t8 + 8 * h;
          const bool hole = PAGED && holes && page_of(key) < 0;
          const uint32_t seen = hole ? 0u : (uint32_t)span;
          const int seen_first = SINKS && !hole ? sink : 0;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            s[n][8 * t8 + i] = (uint32_t)(key + i - first) < seen || (SINKS && key + i < seen_first) ? s[n][8 * t8 + i] : -INFINITY;
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[n][i]);
    top = pair_max(top) * p.scale_log2;
    if (!__any(top > m + PROB_LAG)) return false;
    const float grown = __builtin_fmaxf(m, top);
    keep = grown == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - grown);
    m = grown;
    l *= keep;
    return true;
  };
  // o += the product of tile t's probabilities and values.
  auto product = [&](int t) __attribute__((always_inline)) {
    const uint8_t *vb = lds + (t & 1) * G::BUF + G::K_BYTES + col * 16;
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int t8 = 0; t8 < 2; ++t8)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const u32x4_t a = *(const u32x4_t *)(vb + ((4 * n + 2 * t8 + h) * D + 32 * d) * 16);
          o[d] = mfma32<BF16>(a, pr[n][t8], o[d]);
        }
  };
  // Probabilities, rounded to the type for the product; the sum takes them unrounded.
  auto weigh = [&]() __attribute__((always_inline)) {
    const float base = prob_base<BF16>(m);
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int t8 = 0; t8 < 2; ++t8) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][8 * t8 + i], p.scale_log2, -base));
          l += e[i];
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) pr[n][t8][y] = Half<BF16>::pack(e[2 * y], e[2 * y + 1]);
      }
  };
  // product(t) with weigh() of the next tile and the loads beside it: in each
  // step a product, and of the vector work one group's scores scaled, the last
  // group's exponentials, and the sum and packing of the one before.
  auto product_and_weigh = [&](int t, auto load) __attribute__((always_inline)) {
    const uint8_t *vb = lds + (t & 1) * G::BUF + G::K_BYTES + col * 16;
    auto read = [&](int x) __attribute__((always_inline)) {  // the values of product x = (2n + t8) * DT + d
      return *(const u32x4_t *)(vb + ((2 * (x / DT) + h) * D + 32 * (x % DT)) * 16);
    };
    u32x4_t ring[READS];
    u32x4_t was[NS][2];
    float f[16 * NS], sum[2] = {0.f, 0.f};
    const float base = prob_base<BF16>(m);
#pragma unroll
    for (int n = 0; n < NS; ++n) was[n][0] = pr[n][0], was[n][1] = pr[n][1];
#pragma unroll
    for (int x = 0; x < AHEAD; ++x) ring[x] = read(x);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int x = 0; x < READS + 2; ++x) {
      if (x + AHEAD < READS) ring[x + AHEAD] = read(x + AHEAD);
      if (x >= 2 && x < 14) load(x - 2);
      if (x < READS) o[x % DT] = mfma32<BF16>(ring[x], was[x / DT / 2][x / DT % 2], o[x % DT]);
#pragma unroll
      for (int g = 0; g < NS; ++g) {
        const int e0 = x * NS + g, e1 = e0 - NS, e2 = e1 - NS;
        if (x < READS) f[e0] = __builtin_fmaf(s[e0 / 16][e0 % 16], p.scale_log2, -base);
        if (x >= 1 && x <= READS) f[e1] = __builtin_amdgcn_exp2f(f[e1]);
        if (x >= 2) {
          sum[e2 & 1] += f[e2];
          if (e2 & 1) pr[e2 / 16][e2 / 8 % 2][e2 / 2 % 4] = Half<BF16>::pack(f[e2 - 1], f[e2]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    l += sum[0] + sum[1];
#pragma unroll
    for (int n = 0; n < NS; ++n) asm volatile("" : "+v"(pr[n][0]), "+v"(pr[n][1]));  // made here, not where they are used
  };

  if (n_tiles > 0) {
    // Turn t reads keys t and values t - 1, and stages keys t + 1 and values t
    // (loaded a turn before, their pages looked up two before) into the buffers
    // that turn t - 1 was the last to read.  Past the last tile nothing is
    // loaded and what is staged is not read.
#pragma unroll
    for (int i = 0; i < 4; ++i) put_k(0, i);
    {
      const auto load = fetch(1, kpg_next, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) load(i);
    }
    kpg_next = key_page(2, ka);
    __syncthreads();
    float keep;
    if (!whole_tile(0)) clean_v(0, vpg);
    score_and_stage(0);
    if (CB < 16 && !whole_tile(0)) finite_v(0);
    {
      const auto load = fetch(2, kpg_next, 1, vpg_next);
#pragma unroll
      for (int i = 0; i < 12; ++i) load(i);
    }
    vpg = vpg_next;
    kpg_next = key_page(3, ka), vpg_next = key_page(2, va);
    settle(0, keep);
    weigh();
    __syncthreads();
    for (int t = 1; t < n_tiles; ++t) {
      if (!whole_tile(t)) clean_v(t, vpg);
      score_and_stage(t);
      if (CB < 16 && !whole_tile(t)) finite_v(t);
      int grew = __builtin_amdgcn_readfirstlane((int)settle(t, keep));
      asm volatile("" : "+s"(grew));  // one block of products and vector work for both cases
      product_and_weigh(t - 1, fetch(t + 2, kpg_next, t + 1, vpg_next));
      vpg = vpg_next;
      kpg_next = key_page(t + 3, ka), vpg_next = key_page(t + 2, va);
      if (grew) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= keep;
      }
      __syncthreads();
    }
    product(n_tiles - 1);
  }
  l = pair_sum(l);

  // ---- results: element 4q + i of product d is dim value_dim(d, q, i); for
  // each run of 8 dims (piece) a lane has all 8
  // piece_of: the piece of the lane's run x; (prod, elem): where its j-th dim is.
  auto piece_of = [](int x, int h) __attribute__((always_inline)) { return D == 64 ? 4 * h + x : 8 * (x >> 2) + 4 * h + (x & 3); };
  auto prod = [](int j) __attribute__((always_inline)) { return D == 64 ? j >> 2 : D == 128 ? j >> 1 : j; };
  auto elem = [](int x, int j) __attribute__((always_inline)) {
    return D == 64 ? 4 * (j & 3) + x : D == 128 ? 4 * (2 * (j & 1) + (x >> 2)) + (x & 3) : x;
  };
  if (n_tiles > 0 && s_odd) {
    // rare: once more over the keys of the tiles that not all rows see whole
#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
      if (whole_tile(t)) continue;
      const int k0 = tile_key(t);
#pragma unroll 1
      for (int key = SINKS ? k0 : max(k0, lo); key < min(k0 + BN, hi); ++key) {
        const int pg = PAGED ? page_of(key) : 0;
        if (pg < 0 || (SINKS && !useful(key))) continue;
        const int64_t slot = ((int64_t)head << p.cache.page_shift) + (key & ps_mask);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int piece = piece_of(x, h);
          uint32_t word[PW];
          float scale = 1.f;
          if constexpr (PAGED) {
            load_words(word, p.cache.v + pg * p.cache.v_page + slot * (D * CB / 8) + piece * CB);
            if constexpr (CB < 16) scale = scale_of(p.cache.v_scale[pg * p.cache.vs_page + slot * (D / 32) + (piece >> 2)]);
          } else {
            load_words(word, (const uint8_t *)(p.v.data + (int64_t)(w.q0 + key) * p.v.token + (int64_t)head * p.v.head + 8 * piece));
          }
          const u32x4_t v = eight<BF16, CB>(word, 0, scale);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float f = Half<BF16>::up((v[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
            o[prod(j)][elem(x, j)] +=
                ((uint32_t)(key - first) < (uint32_t)span || (SINKS && key < sink)) && !__builtin_isfinite(f) ? f : 0.f;
          }
        }
      }
    }
  }
  if constexpr (KIND == ATTN_PREFIX) {
    // Rows pass through the wave's quarter of LDS, 64 dims at a time, so that
    // 256 bytes of a row are stored side by side (a lane's own 16 bytes of 32
    // rows each: 512 workgroups, 34 MB, 5 us more).  The 16 pieces of a row are permuted so that neither
    // side meets a bank twice.
    note_items(p, w, head);
    float *y = state_row<D>(p, w.item, head, 7, 32 * wave);
    if (h == 0 && row < rows) *(float2_t *)(y + col * (STATE_PAD + D)) = (float2_t){m, l};
    float4_t *mine = (float4_t *)(lds + wave * 8192);
    __syncthreads();  // the last tile has been read
#pragma unroll
    for (int part = 0; part < D / 64; ++part) {
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const int x = 4 * part + z;
#pragma unroll
        for (int j = 0; j < 8; j += 4)
          mine[col * 16 + ((2 * (piece_of(x, h) & 7) + j / 4) ^ (col & 15))] =
              (float4_t){o[prod(j)][elem(x, j)], o[prod(j + 1)][elem(x, j + 1)], o[prod(j + 2)][elem(x, j + 2)],
                         o[prod(j + 3)][elem(x, j + 3)]};
      }
      lds_order();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 4), q = lane & 15;
        const float4_t v = mine[r * 16 + (q ^ (r & 15))];
        if (r0 + 32 * wave + r < rows) *(float4_t *)(y + r * (STATE_PAD + D) + STATE_PAD + 64 * part + 4 * q) = v;
      }
      lds_order();
    }
    return;
  }
  if constexpr (KIND == ATTN_OWN) {
    if (w.first > 0 && w.split == 0 && row < rows) {
      const Left left = left_for<D>(p, w, row, head);
      const float before = m;
#pragma unroll 4
      for (int x = 0; x < left.parts; ++x) m = __builtin_fmaxf(m, left.row[x * left.step]);
      const float base = m == -INFINITY ? 0.f : m, keep = __builtin_amdgcn_exp2f(before - base);
      l *= keep;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= keep;
#pragma unroll 1
      for (int x = 0; x < left.parts; ++x) {
        const float *from = left.row + x * left.step;
        const float2_t ml = *(const float2_t *)from;
        const float f = __builtin_amdgcn_exp2f(ml.x - base);
        l += ml.y * f;
#pragma unroll
        for (int y = 0; y < D / 16; ++y)
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4_t v = *(const float4_t *)(from + STATE_PAD + 8 * piece_of(y, h) + j);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[prod(j + i)][elem(y, j + i)] += v[i] * f;
          }
      }
    }
  }
  if (w.splits > 1) {
    // a part: [wave][o register / 4][lane][4], then m and the sum of each row;
    // waves whose rows the tile does not have neither write nor read
    constexpr int PART = R * (D + 2);
    constexpr int OV = 4 * DT;
    const bool any = r0 + 32 * wave < rows;
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
      auto of_row = [&](int x, int which) __attribute__((always_inline)) {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            part_of(x0 + x * step), (R * D + which * R + 32 * wave + col) * 4, 0, ATTN_CPOL_SC1));
      };
#pragma unroll 4
      for (int x = 0; x < count; ++x) m = __builtin_fmaxf(m, of_row(x, 0));
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 1
      for (int x = 0; x < count; ++x) {
        const auto rs = part_of(x0 + x * step);
        const float f = __builtin_amdgcn_exp2f(of_row(x, 0) - base);
        l += f * of_row(x, 1);
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
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key is zero
  int ln = lane;
  asm volatile("" : "+v"(ln));  // addresses made here, not held through the loop
  const int64_t own = row_offset(p.out, ln & 31);
  __syncthreads();  // the last tile has been read
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = Half<BF16>::pack(o[prod(2 * j)][elem(x, 2 * j)] * inv, o[prod(2 * j + 1)][elem(x, 2 * j + 1)] * inv);
    *piece_in_lds(ln & 31, piece_of(x, ln >> 5)) = v;
  }
  lds_order();
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const int r = i * RPI + ln / NC;
    const u32x4_t v = *piece_in_lds(r, ln % NC);
    uint16_t *y = piece_at(p.out, own, i, ln);
    if (r0 + 32 * wave + r < rows) *(u32x4_t *)y = v;
  }
}

}  // namespace exl3
