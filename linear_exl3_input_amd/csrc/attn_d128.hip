// Attention kernels for heads of 128 values.
#define EXL3_HEAD_DIM 128
#include "attn_instances.hpp"
