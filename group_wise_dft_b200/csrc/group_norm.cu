// Group norm with a pointwise activation, channels last, forward and backward.
//
// x[B][S][F][N]: B items of S positions, F fields of N group slots, the slot
// fastest.  The F fields form G groups of F / G; per (item b, group g)
//     mean = E[x],  var = E[(x - mean)^2]   over the S (F/G) N values,
//     xhat = (x - mean) rstd,  rstd = 1 / sqrt(var + eps),
//     z = gamma_f xhat + beta_f,  y = act(z).
// gamma and beta are constant along the group axis, the statistics do not
// change when the slots are permuted and act is pointwise in the regular
// domain, so the layer commutes with the group (C_N and D8 alike).
// Backward, with dz = dy act'(z) and n = S (F/G) N:
//     dbeta_f = sum dz,  dgamma_f = sum dz xhat,
//     dx = rstd (gamma dz - sum(gamma dz) / n - xhat sum(gamma dz xhat) / n).
//
// Everything is bound by memory.  Two forms:
//  - an item of at most 32 kRowVecs vectors (a token, S = 1, or a tiny map) is
//    one warp's: its values stay in registers, so they are read once, and the
//    variance is the plain two-pass one;
//  - larger items are split into chunks of positions.  A CTA walks its chunk
//    with one thread per vector of channels (memory order, whole lines), every
//    value going into a running mean and sum of squared deviations (no
//    cancellation, whatever the mean), which are joined per group by the
//    pairwise update of Chan, Golub and LeVeque.  A second launch joins the
//    chunks and normalises.
// Statistics, sums and all arithmetic are fp32; every sum has a fixed order.
#include "activations.cuh"
#include "eqlin_internal.cuh"

namespace eqlin {
namespace {

constexpr int kRowVecs = 8;        // vectors a lane of the row kernels holds
constexpr int kRowWarps = 4;       // warps (items in flight) per CTA of the row kernels
constexpr int kColThreads = 512;   // most threads of a chunk kernel
constexpr int kMaxGroups = 2048;

struct GnShape {
  int64_t B, S;
  int F, N, G;
  int L;            // F N, values per position
  int run;          // L / G, values of a group per position
  int vec;          // values per vector
  int chunks;       // per item (chunk kernels)
  int64_t per;      // positions per chunk
};

template <int BYTES> struct VecOf;
template <> struct VecOf<16> { typedef uint4 type; };
template <> struct VecOf<8> { typedef uint2 type; };
template <> struct VecOf<4> { typedef uint32_t type; };
template <> struct VecOf<2> { typedef uint16_t type; };

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T *p, float (&v)[V]) {
  typedef typename VecOf<V * sizeof(T)>::type Q;
  union { Q q; T e[V]; } u;
  u.q = __ldg(reinterpret_cast<const Q *>(p));
#pragma unroll
  for (int k = 0; k < V; ++k) v[k] = to_f32(u.e[k]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
  typedef typename VecOf<V * sizeof(T)>::type Q;
  union { Q q; T e[V]; } u;
#pragma unroll
  for (int k = 0; k < V; ++k) u.e[k] = from_f32<T>(v[k]);
  *reinterpret_cast<Q *>(p) = u.q;
}

__device__ __forceinline__ float slope_any(int act, float z) {
  float unused;
  return eqlin::slope_any(act, z, unused);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// gamma (or beta) of the V values at channel offset c0, one per SEG values
// (SEG divides N and V, so a segment lies within a field).
template <typename T, int V, int SEG>
__device__ __forceinline__ void load_affine(const T *p, int c0, int N, float missing, float (&a)[V / SEG]) {
#pragma unroll
  for (int k = 0; k < V / SEG; ++k) a[k] = p ? to_f32(__ldg(p + (c0 + k * SEG) / N)) : missing;
}

// ------------------------------------------------------------ row kernels

// Per-group sums of one item: part[q] (shared memory, one value per vector of
// the item) -> out[g] (shared memory).  A team of 32 / ceil_pow2(G) lanes per
// group (one lane per group for G >= 32) walks the group's vectors.
__device__ __forceinline__ void group_sums(const float *part, float *out, const GnShape &sh, int lane) {
  const int runv = sh.run / sh.vec, Lv = sh.L / sh.vec;
  const int count = (int)sh.S * runv;
  int team = 32;
  while (team > 1 && team * sh.G > 32) team >>= 1;
  const int r = lane & (team - 1);
  for (int g0 = 0; g0 < sh.G; g0 += 32 / team) {
    const int g = g0 + lane / team;
    float s = 0.0f;
    if (g < sh.G)
      for (int j = r; j < count; j += team) s += part[(j / runv) * Lv + g * runv + j % runv];
    for (int o = team >> 1; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (g < sh.G && r == 0) out[g] = s;
  }
}

// Shared memory of one warp of a row kernel: a value per vector and two per group.
__host__ __device__ inline int row_smem_floats(const GnShape &sh) {
  return (int)(sh.S * sh.L / sh.vec) + 2 * sh.G;
}

template <typename T, int V, int SEG, int NV>
__global__ void __launch_bounds__(32 * kRowWarps)
group_norm_row_kernel(const T *__restrict__ x, const T *__restrict__ gamma, const T *__restrict__ beta,
                      T *__restrict__ y, float *__restrict__ mean_out, float *__restrict__ rstd_out,
                      GnShape sh, float eps, int act) {
  extern __shared__ float row_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nv = (int)(sh.S * sh.L / V);
  float *part = row_smem + warp * row_smem_floats(sh);
  float *gmean = part + nv, *grstd = gmean + sh.G;
  const int Lv = sh.L / V, runv = sh.run / V;
  const float n = (float)(sh.S * sh.run);
  // a lane's vectors have the same channels in every item: gamma and beta stay in registers
  float ga[NV][V / SEG], be[NV][V / SEG];
  int grp[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int q = lane + 32 * k;
    const int c = q < nv ? q % Lv : 0;
    grp[k] = c / runv;
    load_affine<T, V, SEG>(gamma, c * V, sh.N, 1.0f, ga[k]);
    load_affine<T, V, SEG>(beta, c * V, sh.N, 0.0f, be[k]);
  }
  for (int64_t b = (int64_t)blockIdx.x * kRowWarps + warp; b < sh.B; b += (int64_t)gridDim.x * kRowWarps) {
    const T *src = x + b * sh.S * sh.L;
    float v[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = lane + 32 * k;
      if (q < nv) {
        load_vec<T, V>(src + (int64_t)q * V, v[k]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = 0.0f;
      }
    }
    float m1 = 0.0f, r1 = 0.0f;   // G = 1
    if (sh.G == 1) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) s += v[k][e];
      m1 = warp_sum(s) / n;
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (lane + 32 * k < nv) {
#pragma unroll
          for (int e = 0; e < V; ++e) ss = fmaf(v[k][e] - m1, v[k][e] - m1, ss);
        }
      r1 = rsqrtf(warp_sum(ss) / n + eps);
      if (lane == 0) {
        if (mean_out) mean_out[b] = m1;
        if (rstd_out) rstd_out[b] = r1;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (lane + 32 * k < nv) {
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < V; ++e) s += v[k][e];
          part[lane + 32 * k] = s;
        }
      __syncwarp();
      group_sums(part, gmean, sh, lane);
      __syncwarp();
      for (int g = lane; g < sh.G; g += 32) gmean[g] /= n;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (lane + 32 * k < nv) {
          const float m = gmean[grp[k]];
          float s = 0.0f;
#pragma unroll
          for (int e = 0; e < V; ++e) s = fmaf(v[k][e] - m, v[k][e] - m, s);
          part[lane + 32 * k] = s;
        }
      __syncwarp();
      group_sums(part, grstd, sh, lane);
      __syncwarp();
      for (int g = lane; g < sh.G; g += 32) {
        const float r = rsqrtf(grstd[g] / n + eps);
        grstd[g] = r;
        if (mean_out) mean_out[b * sh.G + g] = gmean[g];
        if (rstd_out) rstd_out[b * sh.G + g] = r;
      }
      __syncwarp();
    }
    T *dst = y + b * sh.S * sh.L;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = lane + 32 * k;
      if (q >= nv) continue;
      const float m = sh.G == 1 ? m1 : gmean[grp[k]], r = sh.G == 1 ? r1 : grstd[grp[k]];
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = act_any(act, fmaf((v[k][e] - m) * r, ga[k][e / SEG], be[k][e / SEG]));
      store_vec<T, V>(dst + (int64_t)q * V, o);
    }
    __syncwarp();   // the next item rewrites part, gmean and grstd
  }
}

// Backward of the row form.  dgamma and dbeta: a lane keeps the sums of its
// segments over the warp's items; at the end the CTA's warps add theirs in
// turn and the CTA writes one partial per field, part[cta][F][2].
template <typename T, int V, int SEG, int NV>
__global__ void __launch_bounds__(32 * kRowWarps)
group_norm_row_backward_kernel(const T *__restrict__ x, const T *__restrict__ dy, const float *__restrict__ mean,
                               const float *__restrict__ rstd, const T *__restrict__ gamma,
                               const T *__restrict__ beta, T *__restrict__ dx, float *__restrict__ part_out,
                               GnShape sh, int act) {
  extern __shared__ float row_smem[];
  constexpr int NS = V / SEG;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nv = (int)(sh.S * sh.L / V);
  float *part = row_smem + warp * row_smem_floats(sh);
  float *c1 = part + nv, *c2 = c1 + sh.G;
  const int Lv = sh.L / V, runv = sh.run / V;
  const float inv_n = 1.0f / (float)(sh.S * sh.run);
  float ga[NV][NS], be[NV][NS], sg[NV][NS], sb[NV][NS];
  int grp[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int q = lane + 32 * k;
    const int c = q < nv ? q % Lv : 0;
    grp[k] = c / runv;
    load_affine<T, V, SEG>(gamma, c * V, sh.N, 1.0f, ga[k]);
    load_affine<T, V, SEG>(beta, c * V, sh.N, 0.0f, be[k]);
#pragma unroll
    for (int j = 0; j < NS; ++j) sg[k][j] = sb[k][j] = 0.0f;
  }
  for (int64_t b = (int64_t)blockIdx.x * kRowWarps + warp; b < sh.B; b += (int64_t)gridDim.x * kRowWarps) {
    const int64_t off = b * sh.S * sh.L;
    // v: x, then xhat; d: dy, then gamma dz
    float v[NV][V], d[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = lane + 32 * k;
      if (q < nv) {
        load_vec<T, V>(x + off + (int64_t)q * V, v[k]);
        load_vec<T, V>(dy + off + (int64_t)q * V, d[k]);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = d[k][e] = 0.0f;
      }
    }
    float s1 = 0.0f, s2 = 0.0f;
    float r[NV], p2[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = lane + 32 * k;
      r[k] = p2[k] = 0.0f;
      if (q >= nv) continue;
      const float m = __ldg(mean + b * sh.G + grp[k]);
      r[k] = __ldg(rstd + b * sh.G + grp[k]);
      float a1 = 0.0f, a2 = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (v[k][e] - m) * r[k];
        float dz = d[k][e];
        if (act != EQLIN_ACT_NONE) dz *= slope_any(act, fmaf(xh, ga[k][e / SEG], be[k][e / SEG]));
        sb[k][e / SEG] += dz;
        sg[k][e / SEG] = fmaf(dz, xh, sg[k][e / SEG]);
        const float dn = dz * ga[k][e / SEG];
        a1 += dn;
        a2 = fmaf(dn, xh, a2);
        v[k][e] = xh;
        d[k][e] = dn;
      }
      s1 += a1;
      s2 += a2;
      p2[k] = a2;
      if (sh.G > 1) part[q] = a1;
    }
    if (sh.G == 1) {
      s1 = warp_sum(s1) * inv_n;
      s2 = warp_sum(s2) * inv_n;
    } else {
      __syncwarp();
      group_sums(part, c1, sh, lane);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (lane + 32 * k < nv) part[lane + 32 * k] = p2[k];
      __syncwarp();
      group_sums(part, c2, sh, lane);
      __syncwarp();
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int q = lane + 32 * k;
      if (q >= nv) continue;
      const float m1 = sh.G == 1 ? s1 : c1[grp[k]] * inv_n, m2 = sh.G == 1 ? s2 : c2[grp[k]] * inv_n;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = r[k] * (d[k][e] - m1 - v[k][e] * m2);
      store_vec<T, V>(dx + off + (int64_t)q * V, o);
    }
    __syncwarp();
  }
  if (!part_out) return;   // the same for the whole grid
  // segment sums of the CTA: seg[(q NS + j)], q over the item's vectors
  __syncthreads();
  float *seg_b = row_smem, *seg_g = row_smem + nv * NS;
  for (int w = 0; w < kRowWarps; ++w) {
    if (warp == w) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int q = lane + 32 * k;
        if (q >= nv) continue;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          seg_b[q * NS + j] = w == 0 ? sb[k][j] : seg_b[q * NS + j] + sb[k][j];
          seg_g[q * NS + j] = w == 0 ? sg[k][j] : seg_g[q * NS + j] + sg[k][j];
        }
      }
    }
    __syncthreads();
  }
  const int per_field = sh.N / SEG, per_pos = sh.L / SEG;
  for (int f = threadIdx.x; f < sh.F; f += blockDim.x) {
    float a = 0.0f, c = 0.0f;
    for (int s = 0; s < (int)sh.S; ++s)
      for (int j = 0; j < per_field; ++j) {
        a += seg_b[s * per_pos + f * per_field + j];
        c += seg_g[s * per_pos + f * per_field + j];
      }
    float *dst = part_out + ((int64_t)blockIdx.x * sh.F + f) * 2;
    dst[0] = a;
    dst[1] = c;
  }
}

// ------------------------------------------------------------ chunk kernels

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

// Running statistics of n values.
struct Stats {
  float n, mean, m2;
};
// Chan, Golub and LeVeque (1979), pairwise update.
__device__ __forceinline__ Stats join(const Stats &a, const Stats &b) {
  Stats r;
  r.n = a.n + b.n;
  if (r.n == 0.0f) return a;
  const float d = b.mean - a.mean, w = b.n / r.n;
  r.mean = fmaf(d, w, a.mean);
  r.m2 = a.m2 + fmaf(d * d * a.n, w, b.m2);
  return r;
}
__device__ __forceinline__ Stats warp_join(Stats a) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Stats b;
    b.n = __shfl_down_sync(0xffffffffu, a.n, o);
    b.mean = __shfl_down_sync(0xffffffffu, a.mean, o);
    b.m2 = __shfl_down_sync(0xffffffffu, a.m2, o);
    a = join(a, b);
  }
  return a;   // lane 0
}

// part[(b chunks + chunk) G + g] = statistics of the chunk's values of group g.
template <typename T, int V>
__global__ void __launch_bounds__(kColThreads)
group_norm_stats_kernel(const T *__restrict__ x, float4 *__restrict__ part, GnShape sh) {
  extern __shared__ float col_smem[];
  const Tiling tl = col_tiling(sh);
  Stats *ts = reinterpret_cast<Stats *>(col_smem);          // [threads]
  Stats *gs = ts + tl.threads;                               // [G]
  const int64_t b = blockIdx.x / sh.chunks;
  const int chunk = (int)(blockIdx.x % sh.chunks);
  const int64_t s0 = chunk * sh.per, s1 = s0 + sh.per < sh.S ? s0 + sh.per : sh.S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarps = blockDim.x >> 5;
  const int Lv = sh.L / V, runv = sh.run / V;
  const int pl = tid / tl.tile, col0 = tid % tl.tile;
  for (int g = tid; g < sh.G; g += blockDim.x) gs[g] = Stats{0.0f, 0.0f, 0.0f};
  for (int t = 0; t < tl.tiles; ++t) {
    const int col = t * tl.tile + col0;
    float mean[V], m2[V], n = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) mean[e] = m2[e] = 0.0f;
    if (pl < tl.lanes && col < Lv) {
      const T *src = x + b * sh.S * sh.L + (int64_t)col * V;
#pragma unroll 4
      for (int64_t s = s0 + pl; s < s1; s += tl.lanes) {
        float v[V];
        load_vec<T, V>(src + s * sh.L, v);
        n += 1.0f;
        const float inv = __fdividef(1.0f, n);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[e] - mean[e];
          mean[e] = fmaf(d, inv, mean[e]);
          m2[e] = fmaf(d, v[e] - mean[e], m2[e]);
        }
      }
    }
    // the vector's values belong to one group: one triple per thread
    Stats st{0.0f, 0.0f, 0.0f};
    if (n > 0.0f) {
      float mu = 0.0f, ss = 0.0f, sp = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) mu += mean[e];
      mu *= 1.0f / V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        ss += m2[e];
        sp = fmaf(mean[e] - mu, mean[e] - mu, sp);
      }
      st = Stats{n * V, mu, fmaf(sp, n, ss)};
    }
    ts[tid] = st;
    __syncthreads();
    // warp w joins the groups w, w + nwarps, ..: the tile's columns of the group, all position lanes
    const int first = t * tl.tile, last = first + tl.tile < Lv ? first + tl.tile : Lv;
    for (int g = first / runv + warp; g <= (last - 1) / runv; g += nwarps) {
      const int a = g * runv > first ? g * runv : first;
      const int z = (g + 1) * runv < last ? (g + 1) * runv : last;
      const int w = z - a, count = w * tl.lanes;
      Stats acc{0.0f, 0.0f, 0.0f};
      for (int j = lane; j < count; j += 32) acc = join(acc, ts[(j / w) * tl.tile + a - first + j % w]);
      acc = warp_join(acc);
      if (lane == 0) gs[g] = join(gs[g], acc);
    }
    __syncthreads();
  }
  for (int g = tid; g < sh.G; g += blockDim.x)
    part[((int64_t)b * sh.chunks + chunk) * sh.G + g] = make_float4(gs[g].n, gs[g].mean, gs[g].m2, 0.0f);
}

template <typename T, int V, int SEG>
__global__ void __launch_bounds__(kColThreads)
group_norm_apply_kernel(const T *__restrict__ x, const T *__restrict__ gamma, const T *__restrict__ beta,
                        const float4 *__restrict__ part, T *__restrict__ y, float *__restrict__ mean_out,
                        float *__restrict__ rstd_out, GnShape sh, float eps, int act) {
  extern __shared__ float col_smem[];
  float2 *gs = reinterpret_cast<float2 *>(col_smem);   // [G] mean, rstd
  const Tiling tl = col_tiling(sh);
  // the last chunks first: what the statistics pass read last is still in L2
  const int64_t unit = (int64_t)gridDim.x - 1 - blockIdx.x;
  const int64_t b = unit / sh.chunks;
  const int chunk = (int)(unit % sh.chunks);
  const int64_t s0 = chunk * sh.per, s1 = s0 + sh.per < sh.S ? s0 + sh.per : sh.S;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nwarps = blockDim.x >> 5;
  for (int g = warp; g < sh.G; g += nwarps) {
    Stats acc{0.0f, 0.0f, 0.0f};
    for (int c = lane; c < sh.chunks; c += 32) {
      const float4 p = __ldg(part + (b * sh.chunks + c) * sh.G + g);
      acc = join(acc, Stats{p.x, p.y, p.z});
    }
    acc = warp_join(acc);
    if (lane == 0) {
      const float r = rsqrtf(acc.m2 / acc.n + eps);
      gs[g] = make_float2(acc.mean, r);
      if (chunk == 0) {
        if (mean_out) mean_out[b * sh.G + g] = acc.mean;
        if (rstd_out) rstd_out[b * sh.G + g] = r;
      }
    }
  }
  __syncthreads();
  const int Lv = sh.L / V, runv = sh.run / V;
  const int pl = tid / tl.tile;
  if (pl >= tl.lanes) return;
  for (int col = tid % tl.tile; col < Lv; col += tl.tile) {
    const float2 mr = gs[col / runv];
    float ga[V / SEG], be[V / SEG];
    load_affine<T, V, SEG>(gamma, col * V, sh.N, 1.0f, ga);
    load_affine<T, V, SEG>(beta, col * V, sh.N, 0.0f, be);
    const int64_t off = b * sh.S * sh.L + (int64_t)col * V;
#pragma unroll 4
    for (int64_t s = s0 + pl; s < s1; s += tl.lanes) {
      float v[V], o[V];
      load_vec<T, V>(x + off + s * sh.L, v);
#pragma unroll
      for (int e = 0; e < V; ++e)
        o[e] = act_any(act, fmaf((v[e] - mr.x) * mr.y, ga[e / SEG], be[e / SEG]));
      store_vec<T, V>(y + off + s * sh.L, o);
    }
  }
}

// Backward, pass 1: part[(b chunks + chunk) F + f] = (sum dz, sum dz xhat) of the chunk.
template <typename T, int V, int SEG>
__global__ void __launch_bounds__(kColThreads)
group_norm_backward_sums_kernel(const T *__restrict__ x, const T *__restrict__ dy, const float *__restrict__ mean,
                                const float *__restrict__ rstd, const T *__restrict__ gamma,
                                const T *__restrict__ beta, float2 *__restrict__ part, GnShape sh, int act) {
  extern __shared__ float col_smem[];
  constexpr int NS = V / SEG;
  float2 *seg = reinterpret_cast<float2 *>(col_smem);   // [lanes][tile NS]
  const Tiling tl = col_tiling(sh);
  const int64_t b = blockIdx.x / sh.chunks;
  const int chunk = (int)(blockIdx.x % sh.chunks);
  const int64_t s0 = chunk * sh.per, s1 = s0 + sh.per < sh.S ? s0 + sh.per : sh.S;
  const int tid = threadIdx.x;
  const int Lv = sh.L / V, runv = sh.run / V;
  const int pl = tid / tl.tile, col0 = tid % tl.tile;
  for (int t = 0; t < tl.tiles; ++t) {
    const int col = t * tl.tile + col0;
    float sb[NS], sg[NS];
#pragma unroll
    for (int j = 0; j < NS; ++j) sb[j] = sg[j] = 0.0f;
    if (pl < tl.lanes && col < Lv) {
      const float m = __ldg(mean + b * sh.G + col / runv), r = __ldg(rstd + b * sh.G + col / runv);
      float ga[NS], be[NS];
      load_affine<T, V, SEG>(gamma, col * V, sh.N, 1.0f, ga);
      load_affine<T, V, SEG>(beta, col * V, sh.N, 0.0f, be);
      const int64_t off = b * sh.S * sh.L + (int64_t)col * V;
#pragma unroll 2
      for (int64_t s = s0 + pl; s < s1; s += tl.lanes) {
        float v[V], d[V];
        load_vec<T, V>(x + off + s * sh.L, v);
        load_vec<T, V>(dy + off + s * sh.L, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (v[e] - m) * r;
          float dz = d[e];
          if (act != EQLIN_ACT_NONE) dz *= slope_any(act, fmaf(xh, ga[e / SEG], be[e / SEG]));
          sb[e / SEG] += dz;
          sg[e / SEG] = fmaf(dz, xh, sg[e / SEG]);
        }
      }
    }
    if (pl < tl.lanes)
#pragma unroll
      for (int j = 0; j < NS; ++j) seg[(pl * tl.tile + col0) * NS + j] = make_float2(sb[j], sg[j]);
    __syncthreads();
    // one thread per field of the tile: its segments, all position lanes
    const int per_field = sh.N / SEG;
    const int first = t * tl.tile, last = first + tl.tile < Lv ? first + tl.tile : Lv;
    const int f0 = (int)((int64_t)first * V / sh.N), nf = (int)((int64_t)(last - first) * V / sh.N);
    for (int f = tid; f < nf; f += blockDim.x) {
      float a = 0.0f, c = 0.0f;
      for (int l = 0; l < tl.lanes; ++l)
        for (int j = 0; j < per_field; ++j) {
          const float2 p = seg[l * tl.tile * NS + f * per_field + j];
          a += p.x;
          c += p.y;
        }
      part[((int64_t)b * sh.chunks + chunk) * sh.F + f0 + f] = make_float2(a, c);
    }
    __syncthreads();
  }
}

// Pass 2, one CTA per item: the chunks' sums in order -> item[b][F] and, with
// gamma, per group c[b][G] = (sum gamma dz, sum gamma dz xhat) / n.
template <typename T>
__global__ void __launch_bounds__(256)
group_norm_backward_item_kernel(const float2 *__restrict__ part, const T *__restrict__ gamma,
                                float2 *__restrict__ item, float2 *__restrict__ c, GnShape sh) {
  const int64_t b = blockIdx.x;
  const int fpg = sh.F / sh.G;
  const float inv_n = 1.0f / ((float)sh.S * (float)sh.run);
  for (int f = threadIdx.x; f < sh.F; f += blockDim.x) {
    float a = 0.0f, q = 0.0f;
    for (int k = 0; k < sh.chunks; ++k) {
      const float2 p = __ldg(part + (b * sh.chunks + k) * sh.F + f);
      a += p.x;
      q += p.y;
    }
    item[b * sh.F + f] = make_float2(a, q);
  }
  __syncthreads();   // the CTA's own global writes are visible to its threads
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int g = warp; g < sh.G; g += blockDim.x >> 5) {
    float a = 0.0f, q = 0.0f;
    for (int j = lane; j < fpg; j += 32) {
      const int f = g * fpg + j;
      const float2 p = item[b * sh.F + f];
      const float w = gamma ? to_f32(gamma[f]) : 1.0f;
      a = fmaf(w, p.x, a);
      q = fmaf(w, p.y, q);
    }
    a = warp_sum(a);
    q = warp_sum(q);
    if (lane == 0) c[b * sh.G + g] = make_float2(a * inv_n, q * inv_n);
  }
}

// dgamma, dbeta from P partials [P][F] of (sum dz, sum dz xhat): 32 fields per
// CTA, 8 threads per field.
template <typename T>
__global__ void __launch_bounds__(256)
group_norm_affine_grad_kernel(const float2 *__restrict__ part, int64_t P, int F, T *__restrict__ dgamma,
                              T *__restrict__ dbeta) {
  __shared__ float2 acc[8][32];
  const int fl = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int f = blockIdx.x * 32 + fl;
  float a = 0.0f, q = 0.0f;
  if (f < F) {
#pragma unroll 4
    for (int64_t p = r; p < P; p += 8) {
      const float2 v = __ldg(part + p * F + f);
      a += v.x;
      q += v.y;
    }
  }
  acc[r][fl] = make_float2(a, q);
  __syncthreads();
  if (r == 0 && f < F) {
    for (int k = 1; k < 8; ++k) {
      a += acc[k][fl].x;
      q += acc[k][fl].y;
    }
    if (dbeta) dbeta[f] = from_f32<T>(a);
    if (dgamma) dgamma[f] = from_f32<T>(q);
  }
}

// Pass 3: dx.
template <typename T, int V, int SEG>
__global__ void __launch_bounds__(kColThreads)
group_norm_backward_apply_kernel(const T *__restrict__ x, const T *__restrict__ dy, const float *__restrict__ mean,
                                 const float *__restrict__ rstd, const T *__restrict__ gamma,
                                 const T *__restrict__ beta, const float2 *__restrict__ c, T *__restrict__ dx,
                                 GnShape sh, int act) {
  const Tiling tl = col_tiling(sh);
  const int64_t unit = (int64_t)gridDim.x - 1 - blockIdx.x;   // as in the forward
  const int64_t b = unit / sh.chunks;
  const int chunk = (int)(unit % sh.chunks);
  const int64_t s0 = chunk * sh.per, s1 = s0 + sh.per < sh.S ? s0 + sh.per : sh.S;
  const int Lv = sh.L / V, runv = sh.run / V;
  const int pl = threadIdx.x / tl.tile;
  if (pl >= tl.lanes) return;
  for (int col = threadIdx.x % tl.tile; col < Lv; col += tl.tile) {
    const int g = col / runv;
    const float m = __ldg(mean + b * sh.G + g), r = __ldg(rstd + b * sh.G + g);
    const float2 cc = __ldg(c + b * sh.G + g);
    float ga[V / SEG], be[V / SEG];
    load_affine<T, V, SEG>(gamma, col * V, sh.N, 1.0f, ga);
    load_affine<T, V, SEG>(beta, col * V, sh.N, 0.0f, be);
    const int64_t off = b * sh.S * sh.L + (int64_t)col * V;
#pragma unroll 2
    for (int64_t s = s0 + pl; s < s1; s += tl.lanes) {
      float v[V], d[V], o[V];
      load_vec<T, V>(x + off + s * sh.L, v);
      load_vec<T, V>(dy + off + s * sh.L, d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = (v[e] - m) * r;
        float dz = d[e];
        if (act != EQLIN_ACT_NONE) dz *= slope_any(act, fmaf(xh, ga[e / SEG], be[e / SEG]));
        o[e] = r * (fmaf(dz, ga[e / SEG], -cc.x) - xh * cc.y);
      }
      store_vec<T, V>(dx + off + s * sh.L, o);
    }
  }
}

// ------------------------------------------------------------ host side

int gcd(int a, int b) {
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

int elem_size(int dtype) { return dtype == EQLIN_F32 ? 4 : 2; }

// Items of at most this many vectors take the row kernels: full-width vectors
// only, since a lane's 8 narrow ones would hold too little to be worth a warp.
bool row_form(const GnShape &sh) { return sh.S * sh.L / sh.vec <= 32 * kRowVecs; }

constexpr int kRowCtas = 148 * 8;   // CTAs of the row kernels (resident at once; also the partials of dgamma, dbeta)
constexpr int64_t kChunkTarget = 148 * 6;   // CTAs that the chunk kernels aim at

int make_shape(int64_t B, int64_t S, int F, int N, int G, int dtype, GnShape *out) {
  if (dtype != EQLIN_F32 && dtype != EQLIN_BF16 && dtype != EQLIN_F16)
    return set_error(EQLIN_ERR_UNSUPPORTED, "dtype %d is not EQLIN_F32, EQLIN_BF16 or EQLIN_F16", dtype);
  if (N < 1 || N > kMaxN) return set_error(EQLIN_ERR_UNSUPPORTED, "N=%d not in 1..16", N);
  if (B < 0 || S < 0) return set_error(EQLIN_ERR_INVALID_ARG, "B=%lld, S=%lld must be >= 0", (long long)B, (long long)S);
  if (F < 1 || G < 1 || F % G != 0)
    return set_error(EQLIN_ERR_INVALID_ARG, "F=%d must be a positive multiple of G=%d", F, G);
  if ((int64_t)F * N > (1 << 24)) return set_error(EQLIN_ERR_UNSUPPORTED, "channel count too large");
  if (G > kMaxGroups) return set_error(EQLIN_ERR_UNSUPPORTED, "G=%d exceeds %d groups", G, kMaxGroups);
  GnShape sh{};
  sh.B = B;
  sh.S = S;
  sh.F = F;
  sh.N = N;
  sh.G = G;
  sh.L = F * N;
  sh.run = sh.L / G;
  if (B > ((int64_t)1 << 40) || S > ((int64_t)1 << 40) || (S > 0 && B > ((int64_t)1 << 46) / S) ||
      (B > 0 && S > 0 && B * S > ((int64_t)1 << 60) / sh.L))
    return set_error(EQLIN_ERR_UNSUPPORTED, "B=%lld items of S=%lld positions are too many", (long long)B, (long long)S);
  // the widest vector that divides a group's values of a position: it never
  // straddles two groups, and every vector is aligned (the base is)
  sh.vec = gcd(sh.run, 16 / elem_size(dtype));
  sh.chunks = 1;
  sh.per = S;
  if (B > 0 && S > 0 && !row_form(sh)) {
    // at least 4 positions per thread and chunk, so that the joining of a
    // chunk stays small beside its loads
    const Tiling tl = col_tiling(sh);
    int64_t want = (kChunkTarget + B - 1) / B;
    const int64_t most = (S + 4 * tl.lanes - 1) / (4 * tl.lanes);
    if (want > most) want = most;
    if (want < 1) want = 1;
    sh.per = (S + want - 1) / want;
    sh.chunks = (int)((S + sh.per - 1) / sh.per);
    if (B * sh.chunks > 0x7fffffffLL)
      return set_error(EQLIN_ERR_UNSUPPORTED, "B=%lld items are too many", (long long)B);
  }
  *out = sh;
  return EQLIN_OK;
}

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

size_t forward_workspace(const GnShape &sh) {
  if (sh.B == 0 || sh.S == 0 || row_form(sh)) return 0;
  return (size_t)sh.B * sh.chunks * sh.G * sizeof(float4);
}

int64_t row_ctas(const GnShape &sh) {
  const int64_t need = (sh.B + kRowWarps - 1) / kRowWarps;
  return need < kRowCtas ? need : kRowCtas;
}

struct BackwardParts {
  size_t part, item, c, total;   // byte offsets
};
BackwardParts backward_parts(const GnShape &sh) {
  BackwardParts p{};
  if (sh.B == 0 || sh.S == 0) return p;
  if (row_form(sh)) {
    p.total = (size_t)row_ctas(sh) * sh.F * sizeof(float2);
    return p;
  }
  p.item = up16((size_t)sh.B * sh.chunks * sh.F * sizeof(float2));
  p.c = p.item + up16((size_t)sh.B * sh.F * sizeof(float2));
  p.total = p.c + (size_t)sh.B * sh.G * sizeof(float2);
  return p;
}

struct Tensors {
  const void *x, *dy, *gamma, *beta;
  void *y;   // or dx
  const float *mean, *rstd;
  float *mean_out, *rstd_out;
  void *dgamma, *dbeta;
};

template <typename T, int V, int SEG, int NV>
int row_forward(const Tensors &t, const GnShape &sh, float eps, int act, cudaStream_t s) {
  const size_t smem = (size_t)kRowWarps * row_smem_floats(sh) * sizeof(float);
  group_norm_row_kernel<T, V, SEG, NV><<<(unsigned)row_ctas(sh), 32 * kRowWarps, smem, s>>>(
      (const T *)t.x, (const T *)t.gamma, (const T *)t.beta, (T *)t.y, t.mean_out, t.rstd_out, sh, eps, act);
  return check_launch("group norm (rows)");
}

template <typename T, int V, int SEG, int NV>
int row_backward(const Tensors &t, const GnShape &sh, int act, float *part, cudaStream_t s) {
  size_t floats = (size_t)kRowWarps * row_smem_floats(sh);
  const size_t segs = 2 * (size_t)(sh.S * sh.L / SEG);
  if (segs > floats) floats = segs;
  group_norm_row_backward_kernel<T, V, SEG, NV><<<(unsigned)row_ctas(sh), 32 * kRowWarps, floats * sizeof(float), s>>>(
      (const T *)t.x, (const T *)t.dy, t.mean, t.rstd, (const T *)t.gamma, (const T *)t.beta, (T *)t.y, part, sh, act);
  return check_launch("group norm backward (rows)");
}

template <typename T, int V, int SEG>
int forward_v(const Tensors &t, const GnShape &sh, float eps, int act, void *ws, cudaStream_t s) {
  if (row_form(sh)) {
    const int nv = (int)(sh.S * sh.L / V);
    if (nv <= 32) return row_forward<T, V, SEG, 1>(t, sh, eps, act, s);
    if (nv <= 96) return row_forward<T, V, SEG, 3>(t, sh, eps, act, s);
    if (nv <= 160) return row_forward<T, V, SEG, 5>(t, sh, eps, act, s);
    return row_forward<T, V, SEG, kRowVecs>(t, sh, eps, act, s);
  }
  const Tiling tl = col_tiling(sh);
  const unsigned grid = (unsigned)(sh.B * sh.chunks);
  float4 *part = static_cast<float4 *>(ws);
  group_norm_stats_kernel<T, V><<<grid, tl.threads, (tl.threads + sh.G) * sizeof(Stats), s>>>((const T *)t.x, part, sh);
  int rc = check_launch("group norm (statistics)");
  if (rc) return rc;
  group_norm_apply_kernel<T, V, SEG><<<grid, tl.threads, sh.G * sizeof(float2), s>>>(
      (const T *)t.x, (const T *)t.gamma, (const T *)t.beta, part, (T *)t.y, t.mean_out, t.rstd_out, sh, eps, act);
  return check_launch("group norm");
}

template <typename T>
int affine_grad(const Tensors &t, const float2 *part, int64_t P, int F, cudaStream_t s) {
  if (!t.dgamma && !t.dbeta) return EQLIN_OK;
  group_norm_affine_grad_kernel<T><<<(unsigned)((F + 31) / 32), 256, 0, s>>>(part, P, F, (T *)t.dgamma, (T *)t.dbeta);
  return check_launch("group norm backward (dgamma, dbeta)");
}

template <typename T, int V, int SEG>
int backward_v(const Tensors &t, const GnShape &sh, int act, void *ws, cudaStream_t s) {
  char *w = static_cast<char *>(ws);
  int rc;
  if (row_form(sh)) {
    const int nv = (int)(sh.S * sh.L / V);
    float *part = t.dgamma || t.dbeta ? reinterpret_cast<float *>(w) : nullptr;
    rc = nv <= 32    ? row_backward<T, V, SEG, 1>(t, sh, act, part, s)
         : nv <= 96  ? row_backward<T, V, SEG, 3>(t, sh, act, part, s)
         : nv <= 160 ? row_backward<T, V, SEG, 5>(t, sh, act, part, s)
                     : row_backward<T, V, SEG, kRowVecs>(t, sh, act, part, s);
    if (rc) return rc;
    return affine_grad<T>(t, reinterpret_cast<const float2 *>(w), row_ctas(sh), sh.F, s);
  }
  const BackwardParts p = backward_parts(sh);
  const Tiling tl = col_tiling(sh);
  const unsigned grid = (unsigned)(sh.B * sh.chunks);
  float2 *part = reinterpret_cast<float2 *>(w + p.part), *item = reinterpret_cast<float2 *>(w + p.item),
         *c = reinterpret_cast<float2 *>(w + p.c);
  group_norm_backward_sums_kernel<T, V, SEG>
      <<<grid, tl.threads, (size_t)tl.lanes * tl.tile * (V / SEG) * sizeof(float2), s>>>(
          (const T *)t.x, (const T *)t.dy, t.mean, t.rstd, (const T *)t.gamma, (const T *)t.beta, part, sh, act);
  if ((rc = check_launch("group norm backward (sums)"))) return rc;
  group_norm_backward_item_kernel<T><<<(unsigned)sh.B, 256, 0, s>>>(part, (const T *)t.gamma, item, c, sh);
  if ((rc = check_launch("group norm backward (items)"))) return rc;
  group_norm_backward_apply_kernel<T, V, SEG><<<grid, tl.threads, 0, s>>>(
      (const T *)t.x, (const T *)t.dy, t.mean, t.rstd, (const T *)t.gamma, (const T *)t.beta, c, (T *)t.y, sh, act);
  if ((rc = check_launch("group norm backward"))) return rc;
  return affine_grad<T>(t, item, sh.B, sh.F, s);
}

// SEG divides N and V: values that share a field.  Full vectors take V or V / 2
// where it divides N; for odd shapes every value looks up its own field.
template <typename T, int V>
int dispatch_seg(bool backward, const Tensors &t, const GnShape &sh, float eps, int act, void *ws, cudaStream_t s) {
  if constexpr (V * sizeof(T) == 16) {
    if (sh.N % V == 0)
      return backward ? backward_v<T, V, V>(t, sh, act, ws, s) : forward_v<T, V, V>(t, sh, eps, act, ws, s);
    if (sh.N % (V / 2) == 0)
      return backward ? backward_v<T, V, V / 2>(t, sh, act, ws, s) : forward_v<T, V, V / 2>(t, sh, eps, act, ws, s);
  }
  return backward ? backward_v<T, V, 1>(t, sh, act, ws, s) : forward_v<T, V, 1>(t, sh, eps, act, ws, s);
}

template <typename T>
int dispatch_vec(bool backward, const Tensors &t, const GnShape &sh, float eps, int act, void *ws, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (sh.vec == 8) return dispatch_seg<T, 8>(backward, t, sh, eps, act, ws, s);
  }
  if (sh.vec == 4) return dispatch_seg<T, 4>(backward, t, sh, eps, act, ws, s);
  if (sh.vec == 2) return dispatch_seg<T, 2>(backward, t, sh, eps, act, ws, s);
  return dispatch_seg<T, 1>(backward, t, sh, eps, act, ws, s);
}

int dispatch(bool backward, int dtype, const Tensors &t, const GnShape &sh, float eps, int act, void *ws,
             cudaStream_t s) {
  if (dtype == EQLIN_F32) return dispatch_vec<float>(backward, t, sh, eps, act, ws, s);
  if (dtype == EQLIN_F16) return dispatch_vec<__half>(backward, t, sh, eps, act, ws, s);
  return dispatch_vec<__nv_bfloat16>(backward, t, sh, eps, act, ws, s);
}

bool aligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_act(int act) {
  if (act != EQLIN_ACT_NONE && act != EQLIN_ACT_SILU && act != EQLIN_ACT_GELU)
    return set_error(EQLIN_ERR_INVALID_ARG, "unknown activation %d", act);
  return EQLIN_OK;
}

int check_workspace(const void *ws, size_t have, size_t need) {
  if (need > 0 && !ws) return set_error(EQLIN_ERR_INVALID_ARG, "null workspace");
  if (have < need) return set_error(EQLIN_ERR_SIZE, "workspace_bytes=%zu < required %zu", have, need);
  if (ws && !aligned(ws, 16)) return set_error(EQLIN_ERR_ALIGN, "workspace must be 16-byte aligned");
  return EQLIN_OK;
}

}  // namespace
}  // namespace eqlin

using namespace eqlin;

extern "C" {

size_t eqlin_group_norm_workspace_bytes(int64_t B, int64_t S, int F, int N, int G, int dtype) {
  GnShape sh;
  if (make_shape(B, S, F, N, G, dtype, &sh) != EQLIN_OK) return 0;
  return forward_workspace(sh);
}

int eqlin_group_norm(const void *x, const void *gamma, const void *beta, void *y, float *mean, float *rstd,
                     int64_t B, int64_t S, int F, int N, int G, float eps, int act, int dtype, void *workspace,
                     size_t workspace_bytes, eqlin_stream_t stream) {
  clear_error();
  GnShape sh;
  int rc = make_shape(B, S, F, N, G, dtype, &sh);
  if (rc || (rc = check_act(act))) return rc;
  if (!(eps >= 0.0f)) return set_error(EQLIN_ERR_INVALID_ARG, "eps must be >= 0");
  if (B == 0 || S == 0) return EQLIN_OK;
  if (!x || !y) return set_error(EQLIN_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(mean, 16) ||
      !aligned(rstd, 16))
    return set_error(EQLIN_ERR_ALIGN, "x, y, gamma, beta, mean and rstd must be 16-byte aligned");
  if ((rc = check_workspace(workspace, workspace_bytes, forward_workspace(sh)))) return rc;
  Tensors t{};
  t.x = x;
  t.gamma = gamma;
  t.beta = beta;
  t.y = y;
  t.mean_out = mean;
  t.rstd_out = rstd;
  return dispatch(false, dtype, t, sh, eps, act, workspace, (cudaStream_t)stream);
}

size_t eqlin_group_norm_backward_workspace_bytes(int64_t B, int64_t S, int F, int N, int G, int dtype) {
  GnShape sh;
  if (make_shape(B, S, F, N, G, dtype, &sh) != EQLIN_OK) return 0;
  return backward_parts(sh).total;
}

int eqlin_group_norm_backward(const void *x, const void *dy, const float *mean, const float *rstd,
                              const void *gamma, const void *beta, void *dx, void *dgamma, void *dbeta, int64_t B,
                              int64_t S, int F, int N, int G, int act, int dtype, void *workspace,
                              size_t workspace_bytes, eqlin_stream_t stream) {
  clear_error();
  GnShape sh;
  int rc = make_shape(B, S, F, N, G, dtype, &sh);
  if (rc || (rc = check_act(act))) return rc;
  if (!aligned(dgamma, 16) || !aligned(dbeta, 16))
    return set_error(EQLIN_ERR_ALIGN, "dgamma and dbeta must be 16-byte aligned");
  if (B == 0 || S == 0) {   // no values: the sums are empty
    const size_t bytes = (size_t)F * elem_size(dtype);
    if (dgamma && cudaMemsetAsync(dgamma, 0, bytes, (cudaStream_t)stream) != cudaSuccess)
      return check_launch("group norm backward (empty)");
    if (dbeta && cudaMemsetAsync(dbeta, 0, bytes, (cudaStream_t)stream) != cudaSuccess)
      return check_launch("group norm backward (empty)");
    return EQLIN_OK;
  }
  if (!x || !dy || !mean || !rstd || !dx) return set_error(EQLIN_ERR_INVALID_ARG, "null pointer");
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(gamma, 16) || !aligned(beta, 16) ||
      !aligned(mean, 16) || !aligned(rstd, 16))
    return set_error(EQLIN_ERR_ALIGN, "x, dy, dx, gamma, beta, mean and rstd must be 16-byte aligned");
  if ((rc = check_workspace(workspace, workspace_bytes, backward_parts(sh).total))) return rc;
  Tensors t{};
  t.x = x;
  t.dy = dy;
  t.gamma = gamma;
  t.beta = beta;
  t.y = dx;
  t.mean = mean;
  t.rstd = rstd;
  t.dgamma = dgamma;
  t.dbeta = dbeta;
  return dispatch(true, dtype, t, sh, 0.0f, act, workspace, (cudaStream_t)stream);
}

}  // extern "C"
