// Attention kernels for heads of 64 values.
#define EXL3_HEAD_DIM 64
#include "attn_instances.hpp"
