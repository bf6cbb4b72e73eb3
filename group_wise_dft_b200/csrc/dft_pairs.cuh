// Real DFT of N group slots, N in 1..16, on two vectors at once (the lanes of a
// float2), for the kernels that take any N.
#pragma once

#include "eqlin_internal.cuh"
#include "tc_transforms.cuh"

namespace eqlin {

// cos and sin of 2 pi j / N (unit_root: exact at quarter turns), rounded once.
struct Trig {
  float c[kMaxN], s[kMaxN];
};
inline Trig make_trig(int N) {
  Trig t{};
  for (int j = 0; j < N; ++j) {
    double c, s;
    unit_root(j, N, &c, &s);
    t.c[j] = (float)c;
    t.s[j] = (float)s;
  }
  return t;
}

__device__ __forceinline__ float2 fma2s(float2 a, float s, float2 c) { return fma2(a, make_float2(s, s), c); }

// Coordinates [Re X0, Re X1, Im X1, ..] (as DftTables).  Slots h and N - h are
// folded first (Re sees their sum, Im their difference): half the products.
template <int N>
__device__ __forceinline__ void fwd_dft2(const float2 (&x)[N], float2 (&z)[N], const Trig &t) {
  if constexpr (N == 8) {
    fwd_cyclic8(x, z);
  } else {
    constexpr int M = (N - 1) / 2;   // folded slots 1 .. M; complex bins 1 .. M
    float2 e[M + 1], o[M + 1];
#pragma unroll
    for (int h = 1; h <= M; ++h) {
      e[h] = add2(x[h], x[N - h]);
      o[h] = sub2(x[h], x[N - h]);
    }
#pragma unroll
    for (int k = 0; k <= N / 2; ++k) {
      float2 re = x[0], im = make_float2(0.0f, 0.0f);
      if (N % 2 == 0) re = k % 2 ? sub2(re, x[N / 2]) : add2(re, x[N / 2]);
#pragma unroll
      for (int h = 1; h <= M; ++h) {
        re = fma2s(e[h], t.c[(k * h) % N], re);
        im = fma2s(o[h], -t.s[(k * h) % N], im);
      }
      if (k == 0)
        z[0] = re;
      else if (2 * k == N)
        z[N - 1] = re;
      else {
        z[2 * k - 1] = re;
        z[2 * k] = im;
      }
    }
  }
}

// y_g = Y_0 + (-1)^g Y_{N/2} + sum_k Re(Y'_k e^{2 pi i g k / N}), the complex bins
// doubled already and the 1/N in the weights; y_g and y_{N-g} share their sums.
template <int N>
__device__ __forceinline__ void inv_dft2(const float2 (&z)[N], float2 (&y)[N], const Trig &t) {
  if constexpr (N == 8) {
    inv_cyclic8(z, y);
  } else {
    constexpr int M = (N - 1) / 2;
#pragma unroll
    for (int g = 0; g <= N / 2; ++g) {
      float2 a = z[0], b = make_float2(0.0f, 0.0f);
      if (N % 2 == 0) a = g % 2 ? sub2(a, z[N - 1]) : add2(a, z[N - 1]);
#pragma unroll
      for (int k = 1; k <= M; ++k) {
        a = fma2s(z[2 * k - 1], t.c[(k * g) % N], a);
        b = fma2s(z[2 * k], -t.s[(k * g) % N], b);
      }
      if (g == 0 || 2 * g == N)
        y[g] = a;
      else {
        y[g] = add2(a, b);
        y[N - g] = sub2(a, b);
      }
    }
  }
}
// N = 1 and 2 have no complex bin (N = 2: Re X0, Re X1)
template <>
__device__ __forceinline__ void fwd_dft2<1>(const float2 (&x)[1], float2 (&z)[1], const Trig &) { z[0] = x[0]; }
template <>
__device__ __forceinline__ void inv_dft2<1>(const float2 (&z)[1], float2 (&y)[1], const Trig &) { y[0] = z[0]; }
template <>
__device__ __forceinline__ void fwd_dft2<2>(const float2 (&x)[2], float2 (&z)[2], const Trig &) {
  z[0] = add2(x[0], x[1]);
  z[1] = sub2(x[0], x[1]);
}
template <>
__device__ __forceinline__ void inv_dft2<2>(const float2 (&z)[2], float2 (&y)[2], const Trig &) {
  y[0] = add2(z[0], z[1]);
  y[1] = sub2(z[0], z[1]);
}

}  // namespace eqlin
