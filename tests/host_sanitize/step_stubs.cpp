// Host-only stand-ins for the launchers of the step's operators: each checks
// the launch it is given as the kernels rely on it (grids, divisors, and that
// everything in the workspace is inside it and apart); nothing touches memory.
#include <cstdio>
#include <cstdlib>

#include "../../linear_exl3_input_amd/csrc/attn_launch.hpp"
#include "../../linear_exl3_input_amd/csrc/step_launch.hpp"

extern long g_launches;
long g_sinks[2] = {0, 0}, g_shared[2] = {0, 0}, g_own[2] = {0, 0}, g_rows = 0, g_tables = 0, g_groups = 0;  // [tile kernel]
long g_split = 0;            // launches whose keys are split
uintptr_t g_ws = 0;          // the workspace that calls are given
size_t g_ws_bytes = 0;

namespace {
constexpr size_t COUNTERS = 65536;

void need(bool ok, const char *what) {
  if (!ok) {
    std::fprintf(stderr, "step launch: %s\n", what);
    std::abort();
  }
}

size_t inside(const void *p, size_t bytes, const char *what) {  // the offset where it ends
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  need(a >= g_ws && a + bytes <= g_ws + g_ws_bytes, what);
  return a + bytes - g_ws;
}

size_t g_ints = 0, g_ints_end = 0;  // the groups' arrays of the call

void check_parts(const exl3::AttnParams &p, int columns, int D, size_t end) {
  const int R = columns ? 16 * columns : exl3::ATTN_TILE_ROWS;
  const int64_t items = (int64_t)p.tokens * p.group / R + p.batch + p.target;
  need(p.tokens > 0 && p.batch > 0 && p.group > 0 && p.heads_kv > 0, "sizes");
  need(items * p.heads_kv <= 0x7FFFFFFFl, "grid");
  need(columns >= 0 && columns <= (D == 256 ? 1 : 2), "columns");
  if (p.target > 0) {
    need(p.counters != nullptr && p.part != nullptr, "workspace");
    need((int64_t)p.part_cap * p.heads_kv * 4 <= (int64_t)COUNTERS, "counters");
    need(p.part_cap >= p.target && p.part_min >= 128, "parts");
    const size_t at = inside(p.part, (size_t)p.part_cap * p.heads_kv * R * (D + 2) * 4, "parts in the workspace");
    need(at <= end, "parts apart from what follows");
    ++g_split;
  }
  ++g_launches;
}

void check_groups(const exl3::GroupsParams &p) {
  need(p.groups > 0 && p.groups <= p.batch, "groups");
  const struct {
    const int32_t *at;
    size_t n;
  } arrays[] = {{p.seq_row, (size_t)p.batch + 1}, {p.start, (size_t)p.batch},      {p.of, (size_t)p.batch},
                {p.first, (size_t)p.groups + 1},  {p.row, (size_t)p.groups + 1}, {p.keys, (size_t)p.groups},       {p.lead, (size_t)p.groups},
                {p.tile_at, (size_t)p.batch + 1}};
  size_t before = COUNTERS;
  g_ints = reinterpret_cast<uintptr_t>(p.seq_row) - g_ws;
  for (const auto &a : arrays) {
    need(reinterpret_cast<uintptr_t>(a.at) - g_ws >= before, "arrays apart");
    before = inside(a.at, 4 * a.n, "arrays in the workspace");
  }
  g_ints_end = before;
}
}  // namespace

namespace exl3 {
#define EXL3_STUB(D)                                                                                                   \
  hipError_t launch_attn_sinks_d##D(bool, int, const AttnParams &p, int columns, hipStream_t) {                       \
    need(p.window > 0 && p.causal == 1 && p.sinks >= 0 && p.sink_keys >= p.sinks && p.sink_keys % 128 == 0, "sinks");  \
    need((int64_t)p.window + p.sink_keys + 1024 <= 0x7FFFFFFFl, "spans within 32 bits");                                \
    check_parts(p, columns, D, g_ws_bytes);                                                                            \
    ++g_sinks[columns == 0];                                                                                           \
    return hipSuccess;                                                                                                 \
  }                                                                                                                    \
  hipError_t launch_attn_prefix_d##D(bool, int, const PrefixParams &p, int columns, hipStream_t) {                    \
    check_groups(p.groups);                                                                                            \
    need(p.cu == p.groups.row && p.kv_len == p.groups.keys && p.batch == p.groups.groups, "groups as sequences");      \
    const int R = columns ? 16 * columns : ATTN_TILE_ROWS;                                                             \
    need(columns >= 0 && columns <= (D == 256 ? 1 : 2), "columns");                                                    \
    need(p.causal == 0 && p.window == 0 && p.target > 0 && p.part_min >= 128 && p.table_row != nullptr, "shared");     \
    need(p.part_cap >= (int64_t)p.tokens * p.group / R + p.batch + p.target, "items");                                 \
    need((int64_t)p.part_cap * p.heads_kv <= 0x7FFFFFFFl, "grid");                                                     \
    inside(p.state, (size_t)p.part_cap * p.heads_kv * R * (STATE_PAD + D) * 4, "state in the workspace");              \
    need(reinterpret_cast<uintptr_t>(p.state) - g_ws >= g_ints_end, "state apart from the groups");                    \
    need(inside(p.group_items, 8 * (size_t)p.batch, "items of the groups") <= reinterpret_cast<uintptr_t>(p.state) - g_ws, \
         "items apart from the state");                                                                               \
    ++g_launches, ++g_shared[columns == 0];                                                                            \
    return hipSuccess;                                                                                                 \
  }                                                                                                                    \
  hipError_t launch_attn_own_d##D(bool, int, const AttnParams &p, int columns, hipStream_t) {                         \
    need(p.start != nullptr && p.group_of != nullptr && p.group_row != nullptr && p.causal == 1, "own");               \
    inside(p.state, ((size_t)p.state_items * p.heads_kv << p.state_shift) * (STATE_PAD + D) * 4, "state");            \
    need(p.state_shift == 4 || p.state_shift == 5 || p.state_shift == 7, "rows of the state");                         \
    check_parts(p, columns, D, g_ints);                                                                                \
    need((p.tile_at != nullptr) == (p.batch >= FEW_SEQUENCES) && (p.tile_at == nullptr || p.target == 0), "tiles");    \
    ++g_own[columns == 0];                                                                                             \
    return hipSuccess;                                                                                                 \
  }
EXL3_STUB(64)
EXL3_STUB(128)
EXL3_STUB(256)
hipError_t launch_norm_rows(int D, bool, int, const NormRowsParams &p, hipStream_t) {
  need((int64_t)p.rows.tokens * (p.rows.hq + p.rows.hk + p.rows.hv) < (1ll << 31) && p.rows.tokens > 0, "rows");
  need(p.axes >= 1 && p.axes <= 4, "axes");
  need((p.wq_step == 0 || p.wq_step == D) && (p.wk_step == 0 || p.wk_step == D), "weights");
  ++g_launches, ++g_rows;
  return hipSuccess;
}
hipError_t launch_tables(const TablesParams &p, hipStream_t) {
  need(p.batch >= 0 && p.tokens >= 0 && p.width >= 0 && p.n_free >= 0 && (1 << p.page_shift) >= 16, "tables");
  ++g_launches, ++g_tables;
  return hipSuccess;
}
hipError_t launch_groups(const GroupsParams &p, hipStream_t) {
  need(p.batch >= FEW_SEQUENCES, "sequences");
  check_groups(p);
  ++g_launches, ++g_groups;
  return hipSuccess;
}
}  // namespace exl3
