// Which keys the sequences of a group share.
#include "step_launch.hpp"
#include "attn_device.hpp"

namespace exl3 {

// few_groups for any number of sequences, as a launch of one workgroup: running
// maxima of the offsets, then a wave to a group.  What bounds it is the chain of
// loads and barriers.
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
  hipLaunchKernelGGL(groups_kernel, dim3(1), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace exl3
