// Internal declarations of the gated cyclic feed-forward layer.
#pragma once

#include "eqlin_internal.cuh"

namespace eqlin {

// What a pass of the spectral product kernels does with its outputs.
constexpr int kEpiLinear = 0;   // y[t][o] = p[t][o]
constexpr int kEpiGated = 1;    // h[t][j] = act(p[t][2j]) p[t][2j + 1]
constexpr int kEpiGates = 2;    // from dh[t][j]: dp[t][2j] = dh p[t][2j + 1] act'(p[t][2j]), dp[t][2j + 1] = dh act(p[t][2j])

struct GatedIo {
  const void *x;      // [T][Cin][N]
  const float *Ws;    // fp32 half spectrum Ws[i][c][o] of the layer Cin -> Cout
  const void *dh;     // kEpiGates: [T][Cout / 2][N]
  void *out;          // kEpiLinear and kEpiGates: [T][Cout][N]; kEpiGated: [T][Cout / 2][N]
  int64_t T;
  int Cin, Cout;
};

// CUDA-core forms (gated_simt.cuh), every N in 1..16; T: float, __nv_bfloat16 or __half.
template <typename T>
int launch_gated_simt_t(int epi, const GatedIo &io, int N, int act, cudaStream_t s);
template <>
int launch_gated_simt_t<float>(int epi, const GatedIo &io, int N, int act, cudaStream_t s);
template <>
int launch_gated_simt_t<__nv_bfloat16>(int epi, const GatedIo &io, int N, int act, cudaStream_t s);
template <>
int launch_gated_simt_t<__half>(int epi, const GatedIo &io, int N, int act, cudaStream_t s);

inline int launch_gated_simt(int epi, const GatedIo &io, int N, int act, int dtype, cudaStream_t s) {
  return dtype == EQLIN_F32   ? launch_gated_simt_t<float>(epi, io, N, act, s)
         : dtype == EQLIN_F16 ? launch_gated_simt_t<__half>(epi, io, N, act, s)
                              : launch_gated_simt_t<__nv_bfloat16>(epi, io, N, act, s);
}

}  // namespace eqlin
