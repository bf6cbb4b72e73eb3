// The group norm's kernels for __half.
#define EQLIN_NORM_TYPE __half
#include "group_norm.cuh"
