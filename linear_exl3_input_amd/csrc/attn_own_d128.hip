// Attention kernels of sequences' own keys, heads of 128 values.
#define EXL3_HEAD_DIM 128
#define EXL3_KIND ATTN_OWN
#define EXL3_PACKED 0
#define EXL3_LAUNCH launch_attn_own_d128
#include "attn_kind_instances.hpp"
