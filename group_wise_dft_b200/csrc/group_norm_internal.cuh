// Shapes and splits of the group norm, shared by its entry points and its kernels' units.
#pragma once

#include "eqlin_internal.cuh"

namespace eqlin {

constexpr int kRowWarps = 4;       // warps (items in flight) per CTA of the row kernels
constexpr int kColThreads = 512;   // most threads of a chunk kernel
constexpr int kMaxGroups = 2048;

struct GnShape {
  int64_t B, S;
  int F, N, G;
  int L;            // F N, values per position
  int run;          // L / G, values of a group per position
  int vec;          // values per vector
  int elem;         // bytes of a value
  int chunks;       // per item (chunk kernels)
  int64_t per;      // positions per chunk
};

inline int gcd(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// Vectors a lane of a row kernel holds, at most: more do not fit its registers
// beside gamma, beta and their gradients' sums.
constexpr int kRowVecs = 5;
// The backward leaves two sums per segment (values that share a field) of an item in
// the 48 KB of shared memory that need no opt-in, beside up to 256 bytes of warps' sums.
constexpr int64_t kRowSegments = 6000;

// The warps that hold an item in their registers: the fewest of 1, 2, 4, 8 (16 where
// a vector lies in one field) whose lanes hold kRowVecs vectors each.  0: too large,
// in chunks, and so are items of narrow vectors that one warp does not hold.
// (us on a B200, bf16 with SiLU, rows against chunks, forward and backward: 65536
// tokens of 320 fields of C_8 141 against 1114 and 387 against 1395; 16384 of 1024,
// 131 against 750 and 324 against 834; 16384 of 2000, 270 against 1270 and 633 against
// 1442; 4000 maps of 10 positions x 80 fields 55 against 137 and 119 against 156.)
inline int row_warps_for(const GnShape &sh) {
  const int64_t nv = sh.S * sh.L / sh.vec;
  if (nv <= 32 * kRowVecs) return 1;
  const int seg = gcd(sh.N, sh.vec), most = seg == sh.vec ? 16 : 8;
  if (nv > most * 32 * kRowVecs || sh.S * sh.L / seg > kRowSegments || sh.vec * sh.elem < 8) return 0;
  int w = 2;
  while (nv > w * 32 * kRowVecs) w *= 2;
  return w;
}
inline bool row_form(const GnShape &sh) { return row_warps_for(sh) > 0; }

constexpr int kRowCtas = 148 * 8;          // most CTAs of a backward row kernel (the partials of dgamma, dbeta)

// Shared memory of one item of a row kernel: a value per vector and two per group.
__host__ __device__ inline int row_smem_floats(const GnShape &sh) {
  return (int)(sh.S * sh.L / sh.vec) + 2 * sh.G;
}

inline int64_t row_ctas(const GnShape &sh, int64_t most = kRowCtas) {
  const int64_t need = row_warps_for(sh) > 1 ? sh.B : (sh.B + kRowWarps - 1) / kRowWarps;
  return need < most ? need : most;
}

// The threads of a chunk kernel: `lanes` positions side by side, one thread
// per vector of a position; positions wider than the CTA go tile by tile
// (tile: vectors per tile, a multiple of N unless it is a whole position, so
// that a tile holds whole fields).
struct Tiling {
  int tile, tiles, lanes, threads;
};
__host__ __device__ inline Tiling col_tiling(const GnShape &sh) {
  Tiling t;
  const int Lv = sh.L / sh.vec;
  t.tile = Lv <= kColThreads ? Lv : kColThreads / sh.N * sh.N;
  t.tiles = (Lv + t.tile - 1) / t.tile;
  t.lanes = kColThreads / t.tile;
  t.threads = (t.lanes * t.tile + 31) / 32 * 32;
  return t;
}

inline size_t up16(size_t v) { return (v + 15) / 16 * 16; }

struct BackwardParts {
  size_t field, group, total;   // byte offsets of the partial sums
};
inline BackwardParts backward_parts(const GnShape &sh) {
  BackwardParts p{};
  if (sh.B == 0 || sh.S == 0) return p;
  if (row_form(sh)) {
    p.total = (size_t)row_ctas(sh) * sh.F * sizeof(float2);
    return p;
  }
  p.group = up16((size_t)sh.B * sh.chunks * sh.F * sizeof(float2));
  p.total = p.group + (size_t)sh.B * sh.chunks * sh.G * sizeof(float2);
  return p;
}

struct NormTensors {
  const void *x, *dy, *gamma, *beta;
  void *y;   // or dx
  const float *mean, *rstd;
  float *mean_out, *rstd_out;
  void *dgamma, *dbeta;
};

// The kernels of one type (group_norm.cuh), forward or backward.
template <typename T>
int launch_group_norm_t(bool backward, const NormTensors &t, const GnShape &sh, float eps, int act, void *ws, cudaStream_t s);
template <>
int launch_group_norm_t<float>(bool, const NormTensors &, const GnShape &, float, int, void *, cudaStream_t);
template <>
int launch_group_norm_t<__nv_bfloat16>(bool, const NormTensors &, const GnShape &, float, int, void *, cudaStream_t);
template <>
int launch_group_norm_t<__half>(bool, const NormTensors &, const GnShape &, float, int, void *, cudaStream_t);

}  // namespace eqlin
