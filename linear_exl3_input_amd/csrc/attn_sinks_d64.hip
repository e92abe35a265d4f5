// Attention kernels with first tokens beside a window, heads of 64 values.
#define EXL3_HEAD_DIM 64
#define EXL3_KIND ATTN_SINKS
#define EXL3_PACKED 1
#define EXL3_LAUNCH launch_attn_sinks_d64
#include "attn_kind_instances.hpp"
