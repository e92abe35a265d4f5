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

// 1 / the root mean square of a row, given the lane's 8 values.  Squares of
// bfloat16 values past 2^64 are infinite; such a row is summed again scaled
// down (its eps counts nothing).
template <int D>
__device__ __forceinline__ float inverse_rms(const float (&f)[8], float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss += f[i] * f[i];
  ss = row_sum<D>(ss);
  if (ss < INFINITY) return __builtin_amdgcn_rsqf(ss * (1.f / D) + eps);
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float g = f[i] * 0x1p-70f;
    ss += g * g;
  }
  return __builtin_amdgcn_rsqf(row_sum<D>(ss) * (1.f / D)) * 0x1p-70f;
}

template <bool BF16, int D, int BITS, bool NORM, bool AXES>
__global__ __launch_bounds__(256) void norm_rows_kernel(NormRowsParams np) {
  const RowsParams &p = np.rows;
  constexpr int LPR = D / 8;  // lanes per row
  const int c = threadIdx.x % LPR;
  const int64_t row = (int64_t)workgroup() * (256 / LPR) + threadIdx.x / LPR;
  const int H = p.hq + p.hk + p.hv;
  if (row >= (int64_t)p.tokens * H) return;  // whole rows leave: the lane moves stay within rows
  const uint32_t t = (uint32_t)row / (uint32_t)H;
  int h = (int)((uint32_t)row - t * (uint32_t)H);
  const bool is_q = h < p.hq, is_v = h >= p.hq + p.hk;
  const Rows src = is_q ? p.q : is_v ? p.v : p.k;
  h -= is_q ? 0 : is_v ? p.hq + p.hk : p.hq;
  const uint16_t *x = src.data + (int64_t)t * src.token + (int64_t)h * src.head;
  u32x4_t own = *(const u32x4_t *)(x + 8 * c);
  uint32_t w[4] = {own.x, own.y, own.z, own.w};
  if (!is_v) {
    float f[8];
    eight_floats<BF16>(own, f);
    float inv = 1.f;
    const float *weight = nullptr;
    if constexpr (NORM) {
      inv = inverse_rms<D>(f, np.eps);
      weight = is_q ? np.wq + (int64_t)h * np.wq_step : np.wk + (int64_t)h * np.wk_step;
      float g[8];
      load_floats(weight + 8 * c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * g[i];
    }
    uint32_t nan = 0;  // values whose position is none
    if (8 * c < p.rot) {
      const int half = p.rot >> 1;
      const bool second = !p.interleaved && 8 * c >= half;  // this lane holds the b of its pairs
      const int i0 = p.interleaved ? 4 * c : second ? 8 * c - half : 8 * c;  // the lane's first pair
      float co[8], si[8];
      if constexpr (AXES) {
        int32_t at[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) at[a] = a < np.axes ? p.positions[a * np.axis_stride + t] : 0;
        const uint32_t word = np.axis_of[i0 >> 4] >> (2 * (i0 & 15));
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
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = f[2 * i], b = f[2 * i + 1];
          f[2 * i] = a * co[i] - b * si[i];
          f[2 * i + 1] = b * co[i] + a * si[i];
        }
      } else {
        const int o0 = second ? i0 : i0 + half;
        float g[8];
        eight_floats<BF16>(*(const u32x4_t *)(x + o0), g);
        if constexpr (NORM) {
          float gw[8];
          load_floats(weight + o0, gw);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = g[i] * inv * gw[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * co[i] + g[i] * (second ? si[i] : -si[i]);  // a*cos - b*sin, or b*cos + a*sin
      }
    }
    if (NORM || 8 * c < p.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = Half<BF16>::pack(f[2 * i], f[2 * i + 1]);
        if (nan != 0) {
          constexpr uint32_t QUIET = BF16 ? 0x7FC0u : 0x7E00u;
          if ((nan >> (2 * i)) & 1u) w[i] = (w[i] & 0xFFFF0000u) | QUIET;
          if ((nan >> (2 * i)) & 2u) w[i] = (w[i] & 0xFFFFu) | QUIET << 16;
        }
      }
    }
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

namespace {

template <bool BF16, int D, int BITS>
hipError_t norm_rows_of(const NormRowsParams &p, hipStream_t s) {
  constexpr int RPB = 256 / (D / 8);
  const int64_t rows = (int64_t)p.rows.tokens * (p.rows.hq + p.rows.hk + p.rows.hv);
  const dim3 grid = grid_of((rows + RPB - 1) / RPB), block(256);
  if (p.wq == nullptr)
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, false, true>), grid, block, 0, s, p);
  else if (p.axes > 1)
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, true, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((norm_rows_kernel<BF16, D, BITS, true, false>), grid, block, 0, s, p);
  return hipGetLastError();
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
