// The CUDA-core kernels of the gated layer for f32 (one unit per type: they build side by side).
#define EQLIN_GATED_TYPE float
#include "gated_simt.cuh"
