// Attention kernels of shared keys, heads of 256 values.
#define EXL3_HEAD_DIM 256
#define EXL3_KIND ATTN_PREFIX
#define EXL3_PACKED 0
#define EXL3_LAUNCH launch_attn_prefix_d256
#include "attn_kind_instances.hpp"
