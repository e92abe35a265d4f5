// Which keys the sequences of a group share, where they are too many for few_groups.
#include "step_launch.hpp"
#include "attn_device.hpp"

namespace exl3 {

// Running maxima of the offsets, and the tiles of own keys' rows before each
// sequence, by one workgroup, then a wave to a group: two launches of 5 us, whose
// chains of loads and barriers are what bounds them.  (A wave to a group in the
// first one's workgroup: 500 groups of two 87 us, 2000 361.  4000 sequences in 4
// groups: 9 and 16 us.)
__global__ __launch_bounds__(1024) void rising_kernel(GroupsParams p) {
  constexpr int N = 1024;
  __shared__ int s_top[3][N / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto row_of = [&](int i) { return i <= p.batch ? min(max(p.cu[i], 0), p.tokens) : 0; };
  int row_top = 0, first_top = 0, tiles_before = 0;
  for (int i0 = 0; i0 <= p.batch; i0 += N) {  // (there are at most as many groups)
    const int i = i0 + tid;
    const int next = row_of(i + 1);
    int r = wave_inclusive_max(row_of(i));
    int f = wave_inclusive_max(i <= p.groups ? min(max(p.group_cu[i], 0), p.batch) : 0);
    if (lane == 63) s_top[0][wave] = r, s_top[1][wave] = f;
    __syncthreads();
    r = max(r, row_top), f = max(f, first_top);
#pragma unroll
    for (int w = 0; w < N / 64; ++w) {
      const int a = s_top[0][w], b = s_top[1][w];
      if (w < wave) r = max(r, a), f = max(f, b);
      row_top = max(row_top, a), first_top = max(first_top, b);
    }
    const int tiles = i < p.batch ? (int)(((int64_t)max(next - r, 0) * p.group + p.tile_rows - 1) / p.tile_rows) : 0;
    const int incl = wave_inclusive_sum(tiles);
    if (lane == 63) s_top[2][wave] = incl;
    __syncthreads();
    int before = tiles_before + incl - tiles;
#pragma unroll
    for (int w = 0; w < N / 64; ++w) {
      const int a = s_top[2][w];
      if (w < wave) before += a;
      tiles_before += a;
    }
    if (i <= p.batch) p.seq_row[i] = r, p.tile_at[i] = before;
    if (i <= p.groups) p.first[i] = f;
  }
}

__global__ __launch_bounds__(256) void groups_kernel(GroupsParams p) {
  const int tid = blockIdx.x * 256 + threadIdx.x, lane = threadIdx.x & 63, g = tid >> 6;
  const int step = gridDim.x * 256;
  // sequences of no group
  for (int s = tid; s < p.first[0]; s += step) p.start[s] = 0;
  for (int s = p.first[p.groups] + tid; s < p.batch; s += step) p.start[s] = 0;
  if (g == p.groups && lane == 0) p.row[g] = p.seq_row[p.first[g]];
  if (g >= p.groups) return;
  const int s0 = p.first[g], s1 = p.first[g + 1];
  int before = 0x7FFFFFFF, live = 0, lead = 0x7FFFFFFF;  // keys before the first new token; sequences that have one
  for (int s = s0 + lane; s < s1; s += 64) {
    const int n = p.seq_row[s + 1] - p.seq_row[s];
    if (n > 0) {
      before = min(before, counted_keys(p.kv_len[s]) - n);
      lead = min(lead, s);
      ++live;
    }
  }
  live = wave_sum(live);
  auto least = [](int v) { return 0x7FFFFFFF - __builtin_amdgcn_readlane(wave_inclusive_max(0x7FFFFFFF - max(v, 0)), 63); };
  before = least(before);
  lead = least(lead);
  const int keys = shared_keys(p, p.prefix_len[g], before, live > 1);
  for (int s = s0 + lane; s < s1; s += 64) {
    p.start[s] = keys;
    p.of[s] = g;
  }
  if (lane == 0) {
    p.row[g] = p.seq_row[s0];
    p.keys[g] = keys;
    p.lead[g] = lead;  // (none: keys is 0)
  }
}

hipError_t launch_groups(const GroupsParams &p, hipStream_t s) {
  hipLaunchKernelGGL(rising_kernel, dim3(1), dim3(1024), 0, s, p);
  hipLaunchKernelGGL(groups_kernel, dim3((p.groups + 4) / 4), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace exl3
