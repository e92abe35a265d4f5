// Attention kernels of shared keys, heads of 128 values.
#define EXL3_HEAD_DIM 128
#define EXL3_KIND ATTN_PREFIX
#define EXL3_PACKED 0
#define EXL3_LAUNCH launch_attn_prefix_d128
#include "attn_kind_instances.hpp"
