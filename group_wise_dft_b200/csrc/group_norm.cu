// Host side of the group norm: checks and workspaces; every check happens before a launch.
#include "group_norm_internal.cuh"

namespace eqlin {
namespace {

int elem_size(int dtype) { return dtype == EQLIN_F32 ? 4 : 2; }

constexpr int64_t kChunkResident = 148 * 2;   // CTAs of a chunk kernel that run at once
constexpr int64_t kChunkFixed = 100 << 10;     // a CTA's start and joins, as bytes of its streaming (about 5 us)

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
      (B > 0 && S > 0 && B * S > ((int64_t)1 << 56) / sh.L))
    return set_error(EQLIN_ERR_UNSUPPORTED, "B=%lld items of S=%lld positions are too many", (long long)B, (long long)S);
  // the widest vector that divides a group's values of a position: it never
  // straddles two groups, and every vector is aligned (the base is)
  sh.elem = elem_size(dtype);
  sh.vec = gcd(sh.run, 16 / sh.elem);
  sh.chunks = 1;
  sh.per = S;
  if (B > 0 && S > 0 && !row_form(sh)) {
    // chunks per item: the fewest rounds of resident CTAs, each as long as its
    // positions and the fixed part; at least 4 positions per thread
    const Tiling tl = col_tiling(sh);
    const int64_t most = (S + 4 * tl.lanes - 1) / (4 * tl.lanes), row = (int64_t)sh.L * elem_size(dtype);
    int64_t best = 1;
    double least = -1.0;
    for (int64_t full = 1; full <= 8; ++full) {   // as many chunks as fill `full` rounds
      int64_t c = full * kChunkResident / B;
      c = c < 1 ? 1 : (c > most ? most : c);
      const int64_t rounds = (B * c + kChunkResident - 1) / kChunkResident;
      const double cost = (double)rounds * ((double)((S + c - 1) / c) * (double)row + (double)kChunkFixed);
      if (least < 0.0 || cost < least) {
        least = cost;
        best = c;
      }
    }
    sh.per = (S + best - 1) / best;
    sh.chunks = (int)((S + sh.per - 1) / sh.per);
    if (B * sh.chunks > 0x7fffffffLL)
      return set_error(EQLIN_ERR_UNSUPPORTED, "B=%lld items are too many", (long long)B);
  }
  *out = sh;
  return EQLIN_OK;
}

size_t forward_workspace(const GnShape &sh) {
  if (sh.B == 0 || sh.S == 0 || row_form(sh)) return 0;
  return (size_t)sh.B * sh.chunks * sh.G * sizeof(float4);
}

int dispatch(bool backward, int dtype, const NormTensors &t, const GnShape &sh, float eps, int act, void *ws,
             cudaStream_t s) {
  if (dtype == EQLIN_F32) return launch_group_norm_t<float>(backward, t, sh, eps, act, ws, s);
  if (dtype == EQLIN_F16) return launch_group_norm_t<__half>(backward, t, sh, eps, act, ws, s);
  return launch_group_norm_t<__nv_bfloat16>(backward, t, sh, eps, act, ws, s);
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
  NormTensors t{};
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
  NormTensors t{};
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
