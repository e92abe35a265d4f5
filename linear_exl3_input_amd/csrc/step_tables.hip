// Block tables and slot maps from request lengths.
#include "step_launch.hpp"
#include "attn_device.hpp"

namespace exl3 {

// With off_b = min(T, sum of q_len before b): request b's rows start at off_b,
// it keeps min(q_len_b, T - off_b) of them, and the pages it needs past those it
// has start at the sum of such needs before b.  Two prefix sums over the
// requests; then every row finds its request by bisection.  All of that is one
// workgroup's work of a microsecond, so each workgroup does it for itself, 256
// requests at a time in LDS, and takes its share of the rows and of the new
// pages: one launch, nothing to wait for between workgroups, and no order that
// timing could change.  Table entries that are read lie below those written.
// What bounds it: a launch and the chain of loads and barriers, 2.8 us for 64
// requests of a token each, 5.4 for 300 requests of 79464 rows (1.4 MB).
__global__ __launch_bounds__(STEP_CHUNK) void tables_kernel(TablesParams p) {
  constexpr int N = STEP_CHUNK;
  __shared__ int s_row[N], s_page[N], s_kv[N], s_have[N];  // first row, first new page, tokens and pages before
  __shared__ int s_sum[2][N / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int step = (int)gridDim.x * N;
  const int mask = (1 << p.page_shift) - 1;
  int row = blockIdx.x * N + tid;   // the thread's next row
  int page = blockIdx.x * N + tid;  // and next new page
  const int base = p.taken ? min(max(*p.taken, 0), p.n_free) : 0;
  int rows = 0, pages = 0;  // of the requests before
  int64_t wanted = 0;
  auto ceil_pages = [&](int n) { return min((int)(((uint32_t)n + (uint32_t)mask) >> p.page_shift), p.width); };
  // The last of the N that starts at or before x.
  auto owner = [&](const int (&starts)[N], int x) {
    int at = 0;
#pragma unroll
    for (int half = N / 2; half > 0; half >>= 1)
      if (starts[at + half] <= x) at += half;
    return at;
  };
  auto number = [&](int j) { return base + j < p.n_free ? p.free_pages[base + j] : -1; };  // j: new pages before
  for (int b0 = 0; b0 < p.batch; b0 += N) {
    const int b = b0 + tid;
    int q = 0, kv = 0;
    if (b < p.batch) {
      q = min(max(p.q_len[b], 0), STEP_MAX_ROWS);
      kv = min(max(p.kv_len[b], 0), STEP_MAX_LEN);
    }
    int incl = wave_inclusive_sum(q);
    if (lane == 63) s_sum[0][wave] = incl;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < N / 64; ++w) {
      if (w < wave) incl += s_sum[0][w];
      all += s_sum[0][w];
    }
    const int start = min(rows + incl - q, p.tokens);  // rows <= 2^20 and 256 requests of 2^20: fits
    const int kept = min(q, p.tokens - start);
    const int have = ceil_pages(kv), more = ceil_pages(kv + kept) - have;
    int pincl = wave_inclusive_sum(more);
    if (lane == 63) s_sum[1][wave] = pincl;
    s_row[tid] = start;
    s_kv[tid] = kv;
    s_have[tid] = have;
    __syncthreads();
    int pall = 0;
#pragma unroll
    for (int w = 0; w < N / 64; ++w) {
      if (w < wave) pincl += s_sum[1][w];
      pall += s_sum[1][w];
    }
    s_page[tid] = pages + pincl - more;
    if (blockIdx.x == 0 && b < p.batch) {
      p.cu[b] = start;
      p.kv_out[b] = kv + kept;
    }
    __syncthreads();
    rows = min(rows + all, p.tokens);
    pages += pall;
    wanted += all;
    for (; row < rows; row += step) {
      const int i = owner(s_row, row);
      const int pos = s_kv[i] + row - s_row[i];
      const int at = pos >> p.page_shift;
      const int own = at < s_have[i] ? p.table[(int64_t)(b0 + i) * p.table_stride + at]
                      : at < p.width ? number(s_page[i] + at - s_have[i])
                                     : -1;
      p.positions[row] = pos;
      p.slots[row] = own >= 0 && own < p.pages ? (own << p.page_shift) + (pos & mask) : -1;
    }
    for (; page < pages; page += step) {
      const int i = owner(s_page, page);
      p.table[(int64_t)(b0 + i) * p.table_stride + s_have[i] + page - s_page[i]] = number(page);
    }
    __syncthreads();
  }
  for (; row < p.tokens; row += step) {
    p.positions[row] = 0;
    p.slots[row] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.cu[p.batch] = rows;
    p.counts[0] = (int)min<int64_t>(wanted, 0x7FFFFFFF);
    p.counts[1] = pages;
  }
}

hipError_t launch_tables(const TablesParams &p, hipStream_t s) {
  const int grid = max(1, min((p.tokens + STEP_CHUNK - 1) / STEP_CHUNK, 512));
  hipLaunchKernelGGL(tables_kernel, dim3(grid), dim3(STEP_CHUNK), 0, s, p);
  return hipGetLastError();
}

}  // namespace exl3
