// The CUDA-core kernels of the gated layer for bf16 (one unit per type: they build side by side).
#define EQLIN_GATED_TYPE __nv_bfloat16
#include "gated_simt.cuh"
