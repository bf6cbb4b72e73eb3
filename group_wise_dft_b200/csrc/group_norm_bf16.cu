// The group norm's kernels for __nv_bfloat16.
#define EQLIN_NORM_TYPE __nv_bfloat16
#include "group_norm.cuh"
