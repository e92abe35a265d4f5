// Host threads that make calls with one workspace: the launches of each call
// follow one another.  The launchers are stand-ins that note whose call they
// belong to and give the other threads time to come between.
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <thread>
#include <vector>

#include <hip/hip_runtime.h>

#include "../../linear_exl3_input_amd/csrc/attn_launch.hpp"
#include "../../linear_exl3_input_amd/csrc/exl3_launch.hpp"
#include "../../linear_exl3_input_amd/csrc/step_launch.hpp"
#include "exl3_step.h"

static thread_local int t_call = 0;  // the call that the thread is in
static std::mutex g_mu;
static std::vector<int> g_launched;

static hipError_t note() {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    g_launched.push_back(t_call);
  }
  std::this_thread::sleep_for(std::chrono::microseconds(300));
  return hipSuccess;
}

namespace exl3 {
hipError_t launch_gemm(int, int, int, int, bool, bool, const GemmParams &, dim3, hipStream_t) { return note(); }
hipError_t launch_dequant(int, int, const DecodeParams &, hipStream_t) { return note(); }
hipError_t launch_gemm_dense(bool, const GemmParams &, dim3, int, int, hipStream_t) { return note(); }
hipError_t launch_gemm_table(int, int, const GemmParams &, int, hipStream_t) { return note(); }
hipError_t launch_input_transform(const void *, bool, bool, int32_t, int32_t, const uint16_t *, int32_t, uint16_t *, hipStream_t,
                                  const int32_t *, const int32_t *, int32_t, int32_t, int32_t) {
  return note();
}
hipError_t launch_epilogue(const float *, int32_t, int32_t, int32_t, int32_t, int32_t, const uint16_t *, const uint16_t *, void *,
                           bool, hipStream_t) {
  return note();
}
hipError_t launch_moe_align(const int32_t *, int32_t, int32_t, int32_t, int32_t, int32_t *, int32_t *, int32_t *, hipStream_t) {
  return note();
}
hipError_t launch_moe_combine(const void *, bool, const int32_t *, const float *, int32_t, int32_t, int32_t, void *, hipStream_t) {
  return note();
}
hipError_t launch_debug_decode(int, int, const DecodeParams &, hipStream_t) { return note(); }
hipError_t launch_debug_codebook(int, uint16_t *, hipStream_t) { return note(); }
hipError_t launch_decode_rate(int, int, const DecodeParams &, hipStream_t) { return note(); }
hipError_t launch_stream_read(const void *, size_t, uint32_t *, hipStream_t) { return note(); }
hipError_t launch_mfma_loop(int32_t, uint16_t, float *, hipStream_t) { return note(); }
#define EXL3_STUB(D)                                                                                                       \
  hipError_t launch_attn_small_d##D(bool, int, const AttnParams &, int, hipStream_t) { return note(); }                    \
  hipError_t launch_attn_tile_d##D(bool, int, const AttnParams &, hipStream_t) { return note(); }                          \
  hipError_t launch_attn_sinks_d##D(bool, int, const AttnParams &, int, hipStream_t) { return note(); }                    \
  hipError_t launch_attn_prefix_d##D(bool, int, const PrefixParams &, int, hipStream_t) { return note(); }                 \
  hipError_t launch_attn_own_d##D(bool, int, const AttnParams &, int, hipStream_t) { return note(); }
EXL3_STUB(64)
EXL3_STUB(128)
EXL3_STUB(256)
hipError_t launch_rows(int, bool, int, const RowsParams &, hipStream_t) { return note(); }
hipError_t launch_cache_read(int, bool, int, const ReadParams &, hipStream_t) { return note(); }
hipError_t launch_norm_rows(int, bool, int, const NormRowsParams &, hipStream_t) { return note(); }
hipError_t launch_tables(const TablesParams &, hipStream_t) { return note(); }
hipError_t launch_groups(const GroupsParams &, hipStream_t) { return note(); }
exl3_status linear_in_scratch(const exl3_weight *, const uint16_t *, int32_t, void *, int32_t, void *, size_t, void *, bool);
}  // namespace exl3

extern "C" {
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int) { return *v = 256, hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *s) { return *s = hipStreamCaptureStatusNone, hipSuccess; }
hipError_t hipEventCreate(hipEvent_t *e) { return *e = nullptr, hipSuccess; }
hipError_t hipEventDestroy(hipEvent_t) { return hipSuccess; }
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipEventSynchronize(hipEvent_t) { return hipSuccess; }
hipError_t hipEventElapsedTime(float *ms, hipEvent_t, hipEvent_t) { return *ms = 5.f, hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "stubbed runtime"; }
}

static void *fake(uintptr_t a) { return reinterpret_cast<void *>(a << 40); }
static const int32_t *ints = static_cast<const int32_t *>(fake(5));

// The calls of one turn of a thread, each with all of the workspace.
static int calls(int which) {
  const size_t bytes = (size_t)1 << 36;
  exl3_kv_cache c;
  std::memset(&c, 0, sizeof c);
  c.k = fake(2), c.v = fake(3);
  c.k_scale = c.v_scale = static_cast<uint8_t *>(fake(4));
  c.k_page_bytes = c.v_page_bytes = 8 * 16 * 128;
  c.k_scale_page_bytes = c.v_scale_page_bytes = 8 * 16 * 128 / 32;
  c.pages = 100, c.page_size = 16, c.heads = 8, c.head_dim = 128, c.dtype = EXL3_BF16, c.bits = 8;
  exl3_rows q = {fake(1), 32 * 128, 128, 32}, k = {fake(1), 8 * 128, 128, 8};
  const int32_t shards[] = {4096};
  exl3_weight w;
  std::memset(&w, 0, sizeof w);
  w.trellis = static_cast<const uint16_t *>(fake(7)), w.suh = static_cast<const uint16_t *>(fake(8));
  w.svh = static_cast<const uint16_t *>(fake(9));
  w.K = 4096, w.N = 4096, w.bits = 4, w.codebook = 1, w.n_shards = 1, w.shard_n = shards;
  const uint16_t *x = static_cast<const uint16_t *>(fake(10));
  void *ws = fake(6), *y = fake(11);
  switch (which) {
    case 0:  // two launches
      return exl3_prefix_attention(&c, &q, &q, ints, ints, ints, 4000, 4000, 16, 16, ints, ints, 1, 0.1f, ws, bytes, nullptr);
    case 1:  // three
      return exl3_prefix_attention(&c, &q, &q, ints, ints, ints, 4000, 4000, 300, 300, ints, ints, 2, 0.1f, ws, bytes, nullptr);
    case 2:
      return exl3_paged_attention(&c, &q, &q, ints, ints, ints, 4000, 4000, 2, 2, 0.1f, 0, ws, bytes, nullptr);
    case 3:
      return exl3_paged_attention_sinks(&c, &q, &q, ints, ints, ints, 4000, 4000, 2, 2, 0.1f, 100, 4, ws, bytes, nullptr);
    case 4:
      return exl3_prompt_attention(&q, &k, &k, &q, ints, 1, 100, 128, EXL3_BF16, 1, 0, 0.1f, ws, bytes, nullptr);
    case 5:
      return exl3_prompt_attention_sinks(&q, &k, &k, &q, ints, 1, 100, 128, EXL3_BF16, 50, 4, 0.1f, ws, bytes, nullptr);
    case 6:
      return exl3_linear(&w, x, 2048, y, EXL3_BF16, ws, bytes, nullptr);
    case 7:
      return exl3_forward(&w, x, EXL3_BF16, 100, y, EXL3_BF16, ws, bytes, nullptr);
    case 8:
      return exl3_moe_linear_ex(&w, 4, x, 64, ints, 16, y, EXL3_BF16, ws, bytes, nullptr, EXL3_DECODER_ALU);
    default:
      return exl3::linear_in_scratch(&w, x, 300, y, EXL3_BF16, ws, (size_t)16 << 20, nullptr, true);
  }
}

int main() {
  constexpr int KINDS = 10, THREADS = 4, TURNS = 6;
  std::atomic<int> bad{0}, next{0};
  int launches[KINDS];
  for (int i = 0; i < KINDS; ++i) {  // how many launches each makes, alone
    g_launched.clear();
    t_call = -1;
    if (calls(i) != EXL3_OK) std::printf("call %d: %s\n", i, exl3_last_error()), ++bad;
    launches[i] = (int)g_launched.size();
    std::printf("call %d: %d launches\n", i, launches[i]);
  }
  g_launched.clear();
  std::vector<std::thread> threads;
  for (int t = 0; t < THREADS; ++t)
    threads.emplace_back([&] {
      for (int i = 0; i < TURNS * KINDS; ++i) {
        t_call = next++;
        if (calls(t_call % KINDS) != EXL3_OK) ++bad;
      }
    });
  for (auto &t : threads) t.join();
  int between = 0, few = 0;
  for (size_t i = 0; i < g_launched.size();) {  // runs of one call's launches
    size_t j = i;
    while (j < g_launched.size() && g_launched[j] == g_launched[i]) ++j;
    if ((int)(j - i) != launches[g_launched[i] % KINDS]) ++between;
    i = j;
  }
  for (int n : {launches[0], launches[1], launches[6], launches[7]}) few += n < 2;  // else this shows nothing
  std::printf("calls with others' launches between: %d, failed: %d, single launches: %d\n", between, (int)bad, few);
  return between != 0 || bad != 0 || few != 0;
}
