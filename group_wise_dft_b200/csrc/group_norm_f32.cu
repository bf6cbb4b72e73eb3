// The group norm's kernels for float.
#define EQLIN_NORM_TYPE float
#include "group_norm.cuh"
