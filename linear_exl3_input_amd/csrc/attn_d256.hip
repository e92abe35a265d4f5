// Attention kernels for heads of 256 values.
#define EXL3_HEAD_DIM 256
#include "attn_instances.hpp"
