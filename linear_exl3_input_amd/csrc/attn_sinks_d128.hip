// Attention kernels with first tokens beside a window, heads of 128 values.
#define EXL3_HEAD_DIM 128
#define EXL3_KIND ATTN_SINKS
#define EXL3_PACKED 1
#define EXL3_LAUNCH launch_attn_sinks_d128
#include "attn_kind_instances.hpp"
