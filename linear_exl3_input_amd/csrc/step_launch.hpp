// Host-side launch interface of the step's tables (include/exl3_step.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn_launch.hpp"

namespace exl3 {

constexpr int32_t STEP_MAX_LEN = 1 << 30;    // what a kv_len counts as at most
constexpr int32_t STEP_MAX_ROWS = 1 << 20;   // what a q_len counts as at most
constexpr int STEP_CHUNK = 256;              // threads of a workgroup, and requests it looks at together

struct TablesParams {
  const int32_t *q_len, *kv_len;
  int32_t *table;
  int64_t table_stride;
  const int32_t *free_pages, *taken;  // taken may be null
  int32_t *cu, *kv_out, *positions, *slots, *counts;
  int32_t batch, tokens, width, pages, page_shift, n_free;
};

hipError_t launch_tables(const TablesParams &p, hipStream_t s);

// What the kernels of shared keys do for themselves for fewer than FEW_SEQUENCES.
hipError_t launch_groups(const GroupsParams &p, hipStream_t s);

}  // namespace exl3
