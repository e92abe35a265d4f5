// Norms of queries and keys for each head and rotary positions of one or
// several axes, in one pass over the rows, with the cache write.
#include "attn_rows.hpp"

namespace exl3 {

// A row x of D values (one token's one head) becomes
//   n = x * rsqrt(mean(x^2) + eps) * w,   then pair i of n's first rot dims
// turns by the angle of position[axis(i)], all in fp32, with one rounding to
// the type at the end.  As in rows_kernel a row is D/8 lanes of one wave with 8
// consecutive values each; the sum of squares goes over those lanes by lane
// moves, and a lane loads its pairs' other halves too where they are rot/2 away.
//
// What bounds it: bytes, with the vector units not far behind (with a row for
// every D/8 lanes and all of the look-up done by lanes, 105 us on the first
// below, 420 vector instructions a wave of two rows, 70% of the cycles; 67 with
// coefficients for several rows; 64 with the look-up as scalar work).
// Measured: 12001 tokens normed, rotated and written to 8 bits, 32/8 heads of
// 128, 270 MB in 64 us, 4.2 TB/s (a copy reaches 4.97); 9973 tokens over three
// axes, 209 MB in 47 us, 4.4 TB/s; 16 tokens, 24/4 heads of 256, 3.1 us.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
  v += lane_xor<1>(v);
  v += lane_xor<2>(v);
  v += lane_xor<4>(v);
  if constexpr (D >= 128) v += lane_xor<8>(v);
  if constexpr (D >= 256) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ void eight_floats(const u32x4_t &w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = Half<BF16>::up(w[i] & 0xFFFFu);
    f[2 * i + 1] = Half<BF16>::up(w[i] >> 16);
  }
}

__device__ __forceinline__ void load_floats(const float *a, float (&f)[8]) {
  const float4_t x = *(const float4_t *)a, y = *(const float4_t *)(a + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = x[i], f[4 + i] = y[i];
}

// 1 / sqrt(x), x positive and normal: the instruction's (within a step of its 24
// bits) and one step of Newton's iteration, without which a whole row's values are
// off the same way by up to that step.  With it, of 49 million values 1150 round to
// the type's other neighbour than in 64 bits; each operation rounded by itself in
// the order norm, weight, rotation: 1550.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  return __builtin_fmaf(0.5f * r, __builtin_fmaf(-x * r, r, 1.f), r);
}

// Of a row's 8 values a lane: 1 / the root of their mean square plus eps.
// Squares of bfloat16 values past 2^64 are infinite; the values of such a row
// are scaled down first, here and in f and g (its eps counts nothing then).
template <int D>
__device__ __forceinline__ float inverse_rms(float (&f)[8], float (&g)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(f[i], f[i], ss);
  ss = row_sum<D>(ss);
  if (ss < INFINITY) return inverse_root(__builtin_fmaf(ss, 1.f / D, eps));
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] *= 0x1p-70f;
    g[i] *= 0x1p-70f;
    ss = __builtin_fmaf(f[i], f[i], ss);
  }
  ss = row_sum<D>(ss) * (1.f / D);
  return ss < INFINITY ? inverse_root(ss) : ss == INFINITY ? 0.f : ss;
}

// A wave has one token and up to 512 / D * HB of its query heads, key heads or
// values: all that is looked up by token, kind and number of heads is then
// scalar work.  What a lane multiplies its values f and their partners g by,
// y = f * A + g * B, depends on the token and the weights alone, so cosines,
// sines and weights are read and multiplied once for HB rows (with norms y is
// multiplied by the row's 1 / rms).
template <bool BF16, int D, int BITS, bool NORM, bool AXES, int HB>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormRowsParams np) {
  const RowsParams &p = np.rows;
  constexpr int LPR = D / 8;     // lanes per row
  constexpr int RPW = 64 / LPR;  // rows side by side
  const int lane = threadIdx.x & 63, c = lane % LPR;
  const int uq = (p.hq + RPW * HB - 1) / (RPW * HB), uk = (p.hk + RPW * HB - 1) / (RPW * HB),
            uv = (p.hv + RPW * HB - 1) / (RPW * HB);
  const int wave = __builtin_amdgcn_readfirstlane(workgroup() * 4 + (threadIdx.x >> 6));
  const int t = quotient(wave, np.by_units);
  if (t >= p.tokens) return;
  int u = wave - t * (uq + uk + uv);
  const bool is_q = u < uq, is_v = u >= uq + uk;
  // (members one by one: a choice between structs puts the arguments into memory)
  auto pick = [&](auto q, auto k, auto v) __attribute__((always_inline)) { return is_q ? q : is_v ? v : k; };
  const int64_t row_step = pick(p.q.head, p.k.head, p.v.head);
  const int heads = pick(p.hq, p.hk, p.hv);
  u -= is_q ? 0 : is_v ? uq + uk : uq;
  const int h0 = u * RPW * HB + lane / LPR;  // the lane's heads h0, h0 + RPW, ...
  const uint16_t *x = pick(p.q.data, p.k.data, p.v.data) + (int64_t)t * pick(p.q.token, p.k.token, p.v.token);
  const int half = p.rot >> 1;
  const bool turns = !is_v && 8 * c < p.rot;
  const bool second = !p.interleaved && 8 * c >= half;  // this lane holds the b of its pairs
  const int i0 = p.interleaved ? 4 * c : second ? 8 * c - half : 8 * c;  // the lane's first pair
  const int o0 = second ? i0 : i0 + half;                                // and its values' partners
  u32x4_t own[HB], other[HB];
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    const uint16_t *row = x + (int64_t)min(h0 + i * RPW, heads - 1) * row_step;
    own[i] = *(const u32x4_t *)(row + 8 * c);
    other[i] = (u32x4_t){0u, 0u, 0u, 0u};
    if (turns && !p.interleaved) other[i] = *(const u32x4_t *)(row + o0);
  }
  float A[8], B[8];
  uint32_t nan = 0;  // values whose position is none
  if (!is_v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) A[i] = 1.f, B[i] = 0.f;
    if (turns) {
      float co[8], si[8];
      if constexpr (AXES) {
        int32_t at[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) at[a] = a < np.axes ? p.positions[a * np.axis_stride + t] : 0;
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) word = i0 >> 4 == i ? np.axis_of[i] : word;
        word >>= 2 * (i0 & 15);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (p.interleaved && i >= 4) break;
          const uint32_t a = (word >> (2 * i)) & 3u;
          const int32_t pos = a & 2u ? (a & 1u ? at[3] : at[2]) : (a & 1u ? at[1] : at[0]);
          const bool known = pos >= 0 && pos < p.n_positions;
          const float2_t v = *(const float2_t *)(p.table + (int64_t)(known ? pos : 0) * p.rot + 2 * (i0 + i));
          co[i] = v.x, si[i] = v.y;
          if (!known) nan |= p.interleaved ? 3u << (2 * i) : 1u << i;
        }
      } else {
        const int32_t pos = p.positions[t];
        const bool known = pos >= 0 && pos < p.n_positions;
        const float *cs = p.table + (int64_t)(known ? pos : 0) * p.rot + 2 * i0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (p.interleaved && i >= 2) break;
          const float4_t v = *(const float4_t *)(cs + 4 * i);
          co[2 * i] = v.x, si[2 * i] = v.y, co[2 * i + 1] = v.z, si[2 * i + 1] = v.w;
        }
        nan = known ? 0u : 0xFFu;
      }
      // a' = a*cos - b*sin, b' = b*cos + a*sin
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          A[2 * i] = A[2 * i + 1] = co[i];
          B[2 * i] = -si[i], B[2 * i + 1] = si[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) A[i] = co[i], B[i] = second ? si[i] : -si[i];
      }
    }
    if constexpr (NORM) {
      const int hw = min(h0, heads - 1);
      const float *weight = is_q ? np.wq + (int64_t)hw * np.wq_step : np.wk + (int64_t)hw * np.wk_step;
      float w[8];
      load_floats(weight + 8 * c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) A[i] *= w[i];
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) B[i] *= w[i ^ 1];
      } else if (turns) {
        load_floats(weight + o0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) B[i] *= w[i];
      }
    }
  }
  int32_t slot_at = -1;
  if constexpr (BITS != 0) {
    if (!is_q) slot_at = p.slots[t];
  }
#pragma unroll
  for (int i = 0; i < HB; ++i) {
    const int h = h0 + i * RPW;
    if (u * RPW * HB + i * RPW >= heads) break;
    uint32_t w[4] = {own[i].x, own[i].y, own[i].z, own[i].w};
    if (!is_v && (NORM || turns)) {
      float f[8], g[8];
      eight_floats<BF16>(own[i], f);
      if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = turns ? f[j ^ 1] : 0.f;  // (B is 0 there, but an infinity times 0 is NaN)
      } else {
        eight_floats<BF16>(other[i], g);
      }
      if constexpr (NORM) {
        const float inv = inverse_rms<D>(f, g, np.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __builtin_fmaf(f[j], A[j], g[j] * B[j]) * inv;
      } else {  // rounded as rows_kernel does
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * A[j] + g[j] * B[j];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = Half<BF16>::pack(f[2 * j], f[2 * j + 1]);
      if (nan != 0) {
        constexpr uint32_t QUIET = BF16 ? 0x7FC0u : 0x7E00u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if ((nan >> (2 * j)) & 1u) w[j] = (w[j] & 0xFFFF0000u) | QUIET;
          if ((nan >> (2 * j)) & 2u) w[j] = (w[j] & 0xFFFFu) | QUIET << 16;
        }
      }
    }
    if (h >= heads) continue;  // whole rows: the lane moves stay within rows
    const u32x4_t res = {w[0], w[1], w[2], w[3]};
    if (is_q) {
      *(u32x4_t *)(p.q_out.data + (int64_t)t * p.q_out.token + (int64_t)h * p.q_out.head + 8 * c) = res;
      continue;
    }
    if (!is_v && p.k_out.data != nullptr)
      *(u32x4_t *)(p.k_out.data + (int64_t)t * p.k_out.token + (int64_t)h * p.k_out.head + 8 * c) = res;
    if constexpr (BITS != 0) {
      const int32_t page = slot_at >> p.cache.page_shift;
      if (slot_at < 0 || page >= p.cache.pages) continue;
      const int off = slot_at & ((1 << p.cache.page_shift) - 1);
      const int64_t r = ((int64_t)h << p.cache.page_shift) + off;  // the row within its page
      uint8_t *codes = is_v ? p.cache.v + page * p.cache.v_page : p.cache.k + page * p.cache.k_page;
      uint8_t *scales = BITS == 16 ? nullptr : is_v ? p.cache.v_scale + page * p.cache.vs_page
                                                    : p.cache.k_scale + page * p.cache.ks_page;
      write_codes<BF16, D, BITS>(w, codes + r * (D * BITS / 8), BITS == 16 ? nullptr : scales + r * (D / 32), c);
    }
  }
}

namespace {

template <bool BF16, int D, int BITS, int HB>
hipError_t norm_rows_heads(NormRowsParams p, hipStream_t s) {
  constexpr int PER = 512 / D * HB;  // heads of a wave
  auto units = [](int heads) { return (heads + PER - 1) / PER; };
  const int each = units(p.rows.hq) + units(p.rows.hk) + units(p.rows.hv);
  p.by_units = Divisor::of((uint32_t)each);
  const dim3 grid = grid_of(((int64_t)p.rows.tokens * each + 3) / 4), block(256);
  if (p.wq == nullptr)
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, false, true, HB>), grid, block, 0, s, p);
  else if (p.axes > 1)
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, true, true, HB>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, true, false, HB>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <bool BF16, int D, int BITS>
hipError_t norm_rows_of(const NormRowsParams &p, hipStream_t s) {
  // Two rows a lane once there are waves enough for it: 32/8/8 heads of 128 in
  // one / two rows a lane, 200 tokens 4.2 / 4.1 us, 500 5.7 / 5.5, 12001 77.7 /
  // 63.7 (four: 4.8, 5.5, 61.7, but over three axes 56.0 where two take 47.2).
  const int64_t waves = (int64_t)p.rows.tokens * (p.rows.hq + p.rows.hk + p.rows.hv) * (D / 8) / 64;
  const bool shared = p.wq_step == 0 && p.wk_step == 0;  // the heads of a lane have the same weights
  return shared && waves >= 4096 ? norm_rows_heads<BF16, D, BITS, 2>(p, s) : norm_rows_heads<BF16, D, BITS, 1>(p, s);
}

template <bool BF16, int D>
hipError_t norm_rows_bits(int bits, const NormRowsParams &p, hipStream_t s) {
  switch (bits) {
    case 0: return norm_rows_of<BF16, D, 0>(p, s);
    case 4: return norm_rows_of<BF16, D, 4>(p, s);
    case 8: return norm_rows_of<BF16, D, 8>(p, s);
    default: return norm_rows_of<BF16, D, 16>(p, s);
  }
}

}  // namespace

hipError_t launch_norm_rows(int head_dim, bool bf16, int bits, const NormRowsParams &p, hipStream_t s) {
  if (bf16)
    return head_dim == 64    ? norm_rows_bits<true, 64>(bits, p, s)
           : head_dim == 128 ? norm_rows_bits<true, 128>(bits, p, s)
                             : norm_rows_bits<true, 256>(bits, p, s);
  return head_dim == 64    ? norm_rows_bits<false, 64>(bits, p, s)
         : head_dim == 128 ? norm_rows_bits<false, 128>(bits, p, s)
                           : norm_rows_bits<false, 256>(bits, p, s);
}

}  // namespace exl3
