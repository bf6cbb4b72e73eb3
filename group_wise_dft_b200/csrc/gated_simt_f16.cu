// The CUDA-core kernels of the gated layer for f16 (one unit per type: they build side by side).
#define EQLIN_GATED_TYPE __half
#include "gated_simt.cuh"
