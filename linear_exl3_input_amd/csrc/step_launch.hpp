// Host-side launch interface of the step's tables (include/exl3_step.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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

// What the two passes of attention with shared prefixes need of the groups.
struct GroupsParams {
  const int32_t *cu, *kv_len;            // [batch+1], [batch]
  const int32_t *group_cu, *prefix_len;  // [groups+1], [groups]
  int32_t batch, tokens, groups, table_keys;
  int32_t *seq_row;                      // [batch+1] the first row of each sequence
  int32_t *start;                        // [batch] the first key that is not shared
  int32_t *first;                        // [groups+1] the first sequence of each group
  int32_t *row;                          // [groups+1] the first row of each group
  int32_t *keys;                         // [groups] its shared keys
  int32_t *of;                           // [batch] the group of each sequence that shares keys
};

hipError_t launch_groups(const GroupsParams &p, hipStream_t s);

}  // namespace exl3
