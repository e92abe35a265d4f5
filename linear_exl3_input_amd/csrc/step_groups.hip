// Which keys the sequences of a group share.
#include "step_launch.hpp"
#include "attn_device.hpp"

namespace exl3 {

// The keys before every new token of a group's sequences, at most prefix_len,
// are read once for all of them.  Rounded down to a multiple of 32, a step of
// the attention kernels, so that neither pass has a step of both.  A group with
// fewer than two sequences that have new tokens shares nothing.
//
// One workgroup: running maxima of the offsets (as find_work has them), then the
// least of each group.  What bounds it is the chain of loads and barriers: 2.7
// us for 4 sequences, 4 to 5 for 64 (from memory, after a large kernel).
__device__ __forceinline__ int shared_keys(const GroupsParams &p, int prefix_len, int before, int live) {
  return live < 2 ? 0 : max(min(min(prefix_len, before), p.table_keys), 0) & ~31;
}

// Fewer than 256 sequences: a thread to each, everything in LDS between one
// round of loads and one of stores.
__global__ __launch_bounds__(256) void few_groups_kernel(GroupsParams p) {
  constexpr int NONE = 0x7FFFFFFF;
  __shared__ int s_row[257], s_first[257], s_before[256], s_live[256], s_top[2][4];
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  const int row = i <= p.batch ? min(max(p.cu[i], 0), p.tokens) : 0;
  const int kv = i < p.batch ? p.kv_len[i] : 0;
  const int seq = i <= p.groups ? min(max(p.group_cu[i], 0), p.batch) : 0;
  const int prefix_len = i < p.groups ? p.prefix_len[i] : 0;
  int r = wave_inclusive_max(row), f = wave_inclusive_max(seq);
  if (lane == 63) s_top[0][wave] = r, s_top[1][wave] = f;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 3; ++w)
    if (w < wave) r = max(r, s_top[0][w]), f = max(f, s_top[1][w]);
  s_row[i] = r;
  s_first[i] = i <= p.groups ? f : NONE;
  s_before[i] = NONE;
  s_live[i] = 0;
  __syncthreads();
  int g = -1;  // the last group that starts at or before the sequence
#pragma unroll
  for (int half = 128; half > 0; half >>= 1)
    if (s_first[g + half] <= i) g += half;
  const bool member = i < p.batch && g >= 0 && i < s_first[p.groups];
  if (member) {
    const int n = s_row[i + 1] - s_row[i];
    if (n > 0) {
      atomicMin(&s_before[g], max(kv, 0) - n);
      atomicAdd(&s_live[g], 1);
    }
  }
  __syncthreads();
  if (i <= p.groups) {
    p.first[i] = f;
    p.row[i] = s_row[f];
    if (i < p.groups) s_before[i] = p.keys[i] = shared_keys(p, prefix_len, s_before[i], s_live[i]);
  }
  __syncthreads();
  if (i < p.batch) {
    p.start[i] = member ? s_before[g] : 0;
    p.of[i] = member ? g : 0;
  }
}

// Any number: a wave to a group.
__global__ __launch_bounds__(256) void groups_kernel(GroupsParams p) {
  __shared__ int s_top[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // to[i] = the largest of from[0..i], each within 0..most
  auto rising = [&](const int32_t *from, int n, int most, int32_t *to) {
    int top = 0;
    for (int i0 = 0; i0 < n; i0 += 256) {
      const int i = i0 + tid;
      int v = wave_inclusive_max(i < n ? min(max(from[i], 0), most) : 0);
      if (lane == 63) s_top[wave] = v;
      __syncthreads();
      v = max(v, top);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (w < wave) v = max(v, s_top[w]);
        top = max(top, s_top[w]);
      }
      if (i < n) to[i] = v;
      __syncthreads();
    }
  };
  rising(p.cu, p.batch + 1, p.tokens, p.seq_row);
  rising(p.group_cu, p.groups + 1, p.batch, p.first);
  // sequences of no group
  for (int s = tid; s < p.first[0]; s += 256) p.start[s] = 0;
  for (int s = p.first[p.groups] + tid; s < p.batch; s += 256) p.start[s] = 0;
  for (int g = wave; g < p.groups; g += 4) {
    const int s0 = p.first[g], s1 = p.first[g + 1];
    int before = 0x7FFFFFFF, live = 0;  // keys before the first new token; sequences that have one
    for (int s = s0 + lane; s < s1; s += 64) {
      const int n = p.seq_row[s + 1] - p.seq_row[s];
      if (n > 0) {
        before = min(before, max(p.kv_len[s], 0) - n);
        ++live;
      }
    }
    live = wave_sum(live);
    before = 0x7FFFFFFF - __builtin_amdgcn_readlane(wave_inclusive_max(0x7FFFFFFF - max(before, 0)), 63);
    const int keys = shared_keys(p, p.prefix_len[g], before, live);
    for (int s = s0 + lane; s < s1; s += 64) {
      p.start[s] = keys;
      p.of[s] = g;
    }
    if (lane == 0) {
      p.row[g] = p.seq_row[s0];
      p.keys[g] = keys;
    }
  }
  if (tid == 0) p.row[p.groups] = p.seq_row[p.first[p.groups]];
}

hipError_t launch_groups(const GroupsParams &p, hipStream_t s) {
  if (p.batch < 256)  // (there are at most as many groups)
    hipLaunchKernelGGL(few_groups_kernel, dim3(1), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(groups_kernel, dim3(1), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace exl3
