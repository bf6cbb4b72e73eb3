// Cyclic C_8 layer with many input fields on tcgen05 tensor cores: the data
// gradient of the gated layer (2H fields -> Cin) and a block's contraction.
//
// y[t,o,:] = sum_i V[o,i,:] * x[t,i,:] (circular convolution over 8 slots) per
// bin of the half spectrum, as in the fused kernel of spectral_tc.cu.  There the
// spectrum of a token tile stays in shared memory while the outputs go by; here
// the input fields are too many for that, so the outputs stay and the inputs go
// by: a CTA pair keeps the accumulators of 128 tokens x up to 128 output fields
// x 8 coordinates in TMEM (512 columns) and walks all input fields once, 16 at
// a time.  The output fields are split into groups of 32..128 (TMEM holds no
// more), and the pairs of a tile's groups run side by side, so that the second
// reading of x comes from L2.
//
// CTA pair (cluster of 2, cta_group::2, instruction M = 128: 64 tokens per CTA),
// one ring of slots; a slot is a K-slice: 16 input fields of 64 tokens (A, 16 KB,
// TMA with the 128-byte swizzle) and their weights for the group (B, 128 co bytes
// per CTA, packed in the order of the shared-memory image).  18 warps per CTA:
//   producer      one thread, TMA of every slot
//   MMA issuer    (leader CTA) 11 MMAs per slot: the real bins 0 and 4 (N = co),
//                 each complex bin as [Im|Re] += Re X . [Wi;Wr] (N = 2 co),
//                 Im += Im X . Wr, Re -= Im X . Wi (N = co, negated B); in the peer
//                 CTA the same warp forwards each transformed slot to the leader's
//                 barrier (one cluster-scope release per slot)
//   16 transform  eight groups of two warps; group s rewrites ring slot s in place
//   warps         (a slot always has the same group, which so sees every phase of
//                 its barrier in order), one thread per token row: 16 fields'
//                 group slots -> coordinates
//   8 of them     are the epilogue too: TMEM -> inverse DFT -> 32-byte stores.  A
//                 unit's accumulators are drained before the next unit's first MMA;
//                 loads and transforms of the ring's slots go on meanwhile.
// Every wait is bounded, as in the other tensor-core kernels.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "gated_internal.cuh"
#include "tc_host.h"
#include "tc_primitives.cuh"
#include "tc_transforms.cuh"

namespace eqlin {
namespace {

constexpr int kThreads = 576;
constexpr int kProd = 0;          // TMA producer; TMEM allocation
constexpr int kMma = 1;           // MMA issuer (leader), forwarder (peer)
constexpr int kTf0 = 2;           // transform warps kTf0 ..
constexpr int kGroups = 8;        // of two warps, one per ring slot
constexpr int kEpi0 = 10;         // the last four groups drain the accumulators too
constexpr int kNumEpi = 8;
static_assert(kTf0 + 2 * kGroups == kThreads / 32 && kEpi0 + kNumEpi == kThreads / 32, "warp roles cover the CTA");

constexpr int kRows = 64;                      // tokens per CTA
constexpr int kTileTokens = 2 * kRows;
constexpr int kBlock = kRows * 128;            // one 8-field block of A
constexpr int kABytes = 2 * kBlock;            // a K-slice of A
constexpr int kMaxSlots = kGroups;
constexpr int kCtrl = 512;
constexpr int kSmemLimit = 232448;
constexpr int kCoMost = 128;                   // output fields per group
constexpr int kCoStep = 32;                    // N = co is a multiple of 32 with cta_group::2
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kSleep = 64;

// Output fields in 32-field blocks, dealt out evenly to the groups (the last
// block may be padding in part: zero weights, no stores).
struct Groups {
  int blocks, n;
  __host__ __device__ explicit Groups(int F_out) {
    blocks = (F_out + kCoStep - 1) / kCoStep;
    n = (blocks * kCoStep + kCoMost - 1) / kCoMost;
  }
  __host__ __device__ int co(int g) const { return kCoStep * (blocks / n + (g < blocks % n ? 1 : 0)); }
  __host__ __device__ int first(int g) const {
    const int r = blocks % n;
    return kCoStep * (g * (blocks / n) + (g < r ? g : r));
  }
};
// One CTA half of a K-slice's weights: panels Re X0, Re X4 [K-chunk 2][co/2 rows][8]
// and bins 1, 2, 3 [K-chunk 2][co rows: Wi of the half's fields, then Wr][8].
__host__ __device__ inline int slice_bytes(int co) { return 128 * co; }
__host__ __device__ inline int panel_at(int k, int co) { return k < 2 ? 16 * co * k : 32 * co * (k - 1); }
__host__ __device__ inline int64_t slice_at(const Groups &gr, int F_in, int g, int jp, int half) {
  return (int64_t)(F_in / 16) * 2 * slice_bytes(1) * gr.first(g) + (int64_t)(2 * jp + half) * slice_bytes(gr.co(g));
}

struct Mma {
  int blk, pair, panel, dgroup, wide, neg, roff;
};
constexpr int kMmas = 11;
// Coordinate c of the half spectrum sits in block c / 4, chunk pair c % 4 of the
// K-slice; TMEM column groups [Re Y0, Re Y4, Im Y1, Re Y1, Im Y2, Re Y2, Im Y3, Re Y3].
__host__ __device__ constexpr Mma mma_of(int f) {
  switch (f) {
    case 0: return {0, 1, 2, 2, 1, 0, 0};    // [Im|Re] Y1 += Re X1 . [Wi;Wr]
    case 1: return {0, 2, 2, 2, 0, 0, 1};    // Im Y1 += Im X1 . Wr
    case 2: return {0, 2, 2, 3, 0, 1, 0};    // Re Y1 -= Im X1 . Wi
    case 3: return {0, 3, 3, 4, 1, 0, 0};    // bin 2: Re = c3, Im = c4
    case 4: return {1, 0, 3, 4, 0, 0, 1};
    case 5: return {1, 0, 3, 5, 0, 1, 0};
    case 6: return {1, 1, 4, 6, 1, 0, 0};    // bin 3: Re = c5, Im = c6
    case 7: return {1, 2, 4, 6, 0, 0, 1};
    case 8: return {1, 2, 4, 7, 0, 1, 0};
    case 9: return {0, 0, 0, 0, 0, 0, 0};    // Re Y0 += Re X0 . W0
    default: return {1, 3, 1, 1, 0, 0, 0};   // Re Y4 += Re X4 . W4
  }
}
// An earlier MMA of the slice already wrote f's columns.
__host__ __device__ constexpr bool accumulates(int f) { return f < 9 && f % 3 != 0; }
__host__ __device__ constexpr int group_coord(int k) {
  return k == 0 ? 0 : k == 1 ? 7 : (k % 2 == 0 ? k : k - 2);
}
static_assert(group_coord(2) == 2 && group_coord(3) == 1 && group_coord(4) == 4 && group_coord(5) == 3 &&
                  group_coord(6) == 6 && group_coord(7) == 5, "Im Y_b is coordinate 2b, Re Y_b is 2b - 1");

struct WideArgs {
  void *y;              // [T][F_out][8], 32-byte aligned
  unsigned int *fault;
  unsigned int epoch;
  int64_t T;
  int F_in, F_out, units, nslots, slot_bytes;
};

// One token's 16 fields (two 128-byte rows: fields 0..7 and 8..15) rewritten in
// place as the coordinates: c of block b at row c / 4, 16-byte chunk 2 (c % 4) + b.
// Row 1's chunks that block 0's coordinates 4..7 overwrite (the even ones) are
// read before they are.
template <bool H>
__device__ __forceinline__ void coords_of(const uint4 (&in)[8], uint32_t (&out)[8][4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float2 x[8], z[8];
    unpack_x8_pair<H>(in[2 * p], in[2 * p + 1], x);
    fwd_cyclic8(x, z);
#pragma unroll
    for (int c = 0; c < 8; ++c) out[c][p] = pack_x2<H>(z[c].x, z[c].y);
  }
}
template <bool H>
__device__ __forceinline__ void transform_row_pair(uint8_t *r0, uint8_t *r1, int sw) {
  uint4 in[8];
  uint32_t out[8][4];
  auto at = [&](int row, int chunk) { return reinterpret_cast<uint4 *>((row ? r1 : r0) + ((chunk ^ sw) << 4)); };
#pragma unroll
  for (int f = 0; f < 8; ++f) in[f] = *at(0, f);
  coords_of<H>(in, out);
#pragma unroll
  for (int f = 0; f < 8; f += 2) in[f] = *at(1, f);
#pragma unroll
  for (int c = 0; c < 8; ++c) *at(c >> 2, 2 * (c & 3)) = make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]);
#pragma unroll
  for (int f = 1; f < 8; f += 2) in[f] = *at(1, f);
  coords_of<H>(in, out);
#pragma unroll
  for (int c = 0; c < 8; ++c) *at(c >> 2, 2 * (c & 3) + 1) = make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]);
}

// TMEM -> y for one warp: lane quarter q4 holds token rows 32 (q4 % 2) .. of this
// CTA and the group's fields of half q4 / 2; the two warps of a quarter take 16
// rows each; a thread has 2 fields x 2 tokens per 8 columns.
template <bool H>
__device__ __noinline__ void wide_epilogue(uint32_t tmem_base, int half, int field0, int64_t tok_base, int64_t T,
                                           int F_out, uint8_t *y, int warp, int lane) {
  using namespace tc;
  const int q4 = warp & 3, h = q4 >> 1, sub = (warp - kEpi0) >> 2;
  const uint32_t tb = tmem_base + ((uint32_t)(q4 * 32 + sub * 16) << 16);
  const int64_t tok0 = tok_base + (q4 & 1) * 32 + sub * 16 + (lane >> 2);
#pragma unroll 1
  for (int fg = 0; fg < half; fg += 8) {
    uint32_t v[8][4];
#pragma unroll
    for (int k = 0; k < 8; ++k) tmem_ld_16x256b(tb + (uint32_t)(k * half + fg), v[k]);
    tmem_wait_ld();
    const int field = field0 + h * half + fg + 2 * (lane & 3);
    // (F_out is a multiple of 8, so a warp's 8 fields are all real or all padding)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float2 z[8], p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        z[group_coord(k)] = make_float2(__uint_as_float(v[k][2 * r]), __uint_as_float(v[k][2 * r + 1]));
      inv_cyclic8(z, p);
      uint32_t a[4], b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        a[q] = pack_x2<H>(p[2 * q].x, p[2 * q + 1].x);
        b[q] = pack_x2<H>(p[2 * q].y, p[2 * q + 1].y);
      }
      const int64_t tok = tok0 + 8 * r;
      if (tok < T && field < F_out) st_global_v8(y + (tok * F_out + field) * 16, a, b);
    }
    __syncwarp();
  }
}

template <bool H>
__global__ void __launch_bounds__(kThreads, 1)
    spectral8_wide_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_big,
                          const __grid_constant__ CUtensorMap map_small, const WideArgs args) {
  using namespace tc;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *const gbase = smem_raw + (base - raw);
  const int nslots = args.nslots;
  const uint32_t slot_bytes = (uint32_t)args.slot_bytes;
  const uint32_t sBar = base + (uint32_t)nslots * slot_bytes;
  auto bar_x = [&](int s) { return sBar + 8u * s; };                       // A landed (this CTA)
  auto bar_b = [&](int s) { return sBar + 8u * (kMaxSlots + s); };         // both halves of B landed (leader)
  auto bar_a = [&](int s) { return sBar + 8u * (2 * kMaxSlots + s); };     // A transformed
  auto bar_empty = [&](int s) { return sBar + 8u * (3 * kMaxSlots + s); }; // the slot's MMAs are done
  const uint32_t bar_acc_full = sBar + 8u * (4 * kMaxSlots);
  const uint32_t bar_acc_empty = sBar + 8u * (4 * kMaxSlots + 1);          // leader
  const uint32_t tmem_slot = sBar + 8u * (4 * kMaxSlots + 2);
  static_assert(8 * (4 * kMaxSlots + 2) + 4 <= kCtrl, "control block");
  volatile uint32_t *tmem_slot_ptr = reinterpret_cast<volatile uint32_t *>(gbase + (tmem_slot - base));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const FaultCtx fault{args.fault, args.epoch};
  const Groups gr(args.F_out);
  const int nst = args.F_in / 16;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(bar_x(s), 1);
      mbar_init(bar_b(s), 1);
      mbar_init(bar_a(s), leader ? 3 : 2);   // a group's two warps (+ the peer's forwarder)
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_acc_full, 1);
    mbar_init(bar_acc_empty, 2 * kNumEpi);
    fence_mbarrier_init_cluster();
  }
  if (warp == kProd) tmem_alloc_pair(tmem_slot, kTmemCols);
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync();
  tcgen05_fence_after();
  const uint32_t tmem_base = *tmem_slot_ptr;

  // unit n of this pair: neighbouring pairs take a tile's groups side by side.
  // Where every round of the pairs takes whole tiles, a pair's group changes
  // from round to round (the groups' sizes differ).
  const int nunits = args.units > pair ? (args.units - pair + npairs - 1) / npairs : 0;
  auto unit_tile = [&](int n) { return (pair + n * npairs) / gr.n; };
  auto unit_group = [&](int n) { return (pair + n * npairs + (npairs % gr.n == 0 ? n : 0)) % gr.n; };

  if (warp == kProd) {
    if (elect_one_sync()) {
      prefetch_tensormap(&map_x);
      prefetch_tensormap(&map_big);
      prefetch_tensormap(&map_small);
      const uint32_t leader_b = mapa_shared(bar_b(0), 0);
      const int co_big = gr.co(0);
      uint32_t s = 0, ph = 0;
      bool ok = true;
      for (int n = 0; n < nunits && ok; ++n) {
        const int g = unit_group(n), co = gr.co(g);
        const int row0 = unit_tile(n) * kTileTokens + (int)rank * kRows;
        const int rows = slice_bytes(co) / 512;
        int brow = (int)(slice_at(gr, args.F_in, g, 0, (int)rank) / 512);
        const void *mb = co == co_big ? &map_big : &map_small;
        for (int jp = 0; jp < nst; ++jp, brow += 2 * rows) {
          if (!mbar_wait_bounded(bar_empty(s), ph ^ 1u, fault, FAULT_WAIT_B_EMPTY, kWaitNs)) {
            ok = false;
            break;
          }
          const uint32_t slot = base + s * slot_bytes;
          mbar_arrive_expect_tx(bar_x(s), (uint32_t)kABytes);
          tma_load_2d(slot, &map_x, bar_x(s), jp * 128, row0);
          tma_load_2d(slot + kBlock, &map_x, bar_x(s), jp * 128 + 64, row0);
          if (leader) mbar_arrive_expect_tx(bar_b(s), 2u * (uint32_t)slice_bytes(co));
          tma_load_2d_pair(slot + kABytes, mb, leader_b + 8u * s, 0, brow);
          if (++s == (uint32_t)nslots) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kMma) {
    uint32_t s = 0, ph = 0;
    bool ok = true;
    if (leader) {
      const uint64_t a0 = smem_desc_kmajor_sw128(base);
      const uint64_t b0 = smem_desc_kmajor_noswizzle(base + kABytes, 0u, 128u);
      const uint32_t a_hi = (uint32_t)(a0 >> 32), b_hi = (uint32_t)(b0 >> 32);
      for (int n = 0; n < nunits && ok; ++n) {
        const int co = gr.co(unit_group(n)), half = co / 2;
        const uint32_t id_n = H ? idesc_f16_f32(128, co) : idesc_bf16_f32(128, co);
        const uint32_t id_w = H ? idesc_f16_f32(128, 2 * co) : idesc_bf16_f32(128, 2 * co);
        uint32_t dm[kMmas], b_lo[kMmas];
#pragma unroll
        for (int f = 0; f < kMmas; ++f) {
          const Mma m = mma_of(f);
          dm[f] = tmem_base + (uint32_t)(m.dgroup * half);
          const int rows = m.panel < 2 ? half : co;       // B rows per K-chunk
          b_lo[f] = (uint32_t)b0 + (uint32_t)((panel_at(m.panel, co) + m.roff * half * 16) >> 4) +
                    ((uint32_t)rows << 16);               // leading byte offset: one K-chunk of rows
        }
        if (!mbar_wait_bounded_warp(bar_acc_empty, ((uint32_t)n & 1u) ^ 1u, fault, FAULT_WAIT_ACC_EMPTY, kWaitNs)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        for (int jp = 0; jp < nst; ++jp) {
          if (!mbar_wait_bounded_warp(bar_a(s), ph, fault, FAULT_WAIT_A_FULL, kWaitNs) ||
              !mbar_wait_bounded_warp(bar_b(s), ph, fault, FAULT_WAIT_B_FULL, kWaitNs)) {
            ok = false;
            break;
          }
          tcgen05_fence_after();
          if (elect_one_sync()) {
            const uint32_t at = s * (slot_bytes >> 4), acc = jp > 0 ? 1u : 0u;
#pragma unroll
            for (int f = 0; f < kMmas; ++f) {
              const Mma m = mma_of(f);
              mma_bf16_pair_w(dm[f], (uint32_t)a0 + at + (uint32_t)(m.blk * (kBlock >> 4) + m.pair * 2), a_hi,
                              b_lo[f] + at, b_hi, (m.wide ? id_w : id_n) | (m.neg ? (1u << 14) : 0u),
                              acc | (accumulates(f) ? 1u : 0u));
            }
            mma_commit_pair_mc(bar_empty(s), 0x3);
          }
          __syncwarp();
          if (++s == (uint32_t)nslots) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one_sync()) mma_commit_pair_mc(bar_acc_full, 0x3);
        __syncwarp();
      }
    } else {
      const uint32_t leader_a = mapa_shared(bar_a(0), 0);
      const int total = nunits * nst;
      for (int q = 0; q < total; ++q) {
        if (!mbar_wait_bounded_warp(bar_a(s), ph, fault, FAULT_WAIT_A_FULL, kWaitNs)) break;
        if (elect_one_sync()) mbar_arrive_cluster(leader_a + 8u * s);
        __syncwarp();
        if (++s == (uint32_t)nslots) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
  } else {
    const int grp = (warp - kTf0) >> 1;
    const int row = ((warp - kTf0) & 1) * 32 + lane;
    const bool epi = warp >= kEpi0;
    const uint32_t leader_acc_empty = mapa_shared(bar_acc_empty, 0);
    int q = grp;                     // this group's next slot use (none past the ring)
    uint32_t ph = 0;
    const uint32_t s = (uint32_t)grp;
    bool ok = true;
    for (int n = 0; n < nunits && ok; ++n) {
      for (const int end = grp < nslots ? (n + 1) * nst : 0; q < end; q += nslots, ph ^= 1u) {
        if (!mbar_wait_bounded(bar_x(s), ph, fault, FAULT_WAIT_X_FULL, kWaitNs, kSleep)) {
          ok = false;
          break;
        }
        uint8_t *r0 = gbase + (size_t)s * slot_bytes + row * 128;
        transform_row_pair<H>(r0, r0 + kBlock, row & 7);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(bar_a(s));
      }
      if (!ok || !epi) continue;
      if (!mbar_wait_bounded(bar_acc_full, (uint32_t)n & 1u, fault, FAULT_WAIT_ACC_FULL, kWaitNs, kSleep)) {
        ok = false;
        break;
      }
      tcgen05_fence_after();
      const int g = unit_group(n);
      wide_epilogue<H>(tmem_base, gr.co(g) / 2, gr.first(g),
                       (int64_t)unit_tile(n) * kTileTokens + (int64_t)rank * kRows, args.T, args.F_out,
                       static_cast<uint8_t *>(args.y), warp, lane);
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(leader_acc_empty);
    }
  }

  __syncwarp();
  if (fault_raised(fault)) {   // give copies still in flight time to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kProd) {
    tcgen05_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// ---------------------------------------------------------------- packing

// One thread per (output field o, 8 input fields): the half spectrum of
// V[o, i, :] = W[i, o, -m] (the adjoint: the conjugate of W[i, o]'s) or W[o, i, m],
// the 1/8 of the inverse DFT and the 2 of its one-sided bins folded in, as one
// 16-byte run of 8 input fields per panel row, and in fp32 as Ws[i][c][o] for the
// CUDA-core kernels.  Lanes walk o, so both stores are coalesced.
template <bool H, bool ADJ>
__global__ void __launch_bounds__(256)
pack_wide_kernel(const uint4 *__restrict__ W, int F_in, int F_out, float *__restrict__ Ws, uint8_t *__restrict__ dst) {
  const Groups gr(F_out);
  const int padded = gr.blocks * kCoStep;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= (int64_t)padded * (F_in / 8)) return;
  const int o = (int)(idx % padded), ib = (int)(idx / padded);
  uint32_t out[8][4];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float2 x[8], z[8];
    const int i = 8 * ib + 2 * p;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (o < F_out) {
      a = __ldg(W + (ADJ ? (size_t)i * F_out + o : (size_t)o * F_in + i));
      b = __ldg(W + (ADJ ? (size_t)(i + 1) * F_out + o : (size_t)o * F_in + i + 1));
    }
    unpack_x8_pair<H>(a, b, x);
    fwd_cyclic8(x, z);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float2 v = scl2(z[c], ADJ && c % 2 == 0 && c > 0 ? -0.125f : 0.125f);   // c = 2, 4, 6: Im
      if (o < F_out) {
        Ws[((size_t)i * 8 + c) * F_out + o] = v.x;
        Ws[((size_t)(i + 1) * 8 + c) * F_out + o] = v.y;
      }
      const float2 t = c == 0 || c == 7 ? v : scl2(v, 2.0f);
      out[c][p] = pack_x2<H>(t.x, t.y);
    }
  }
  int g = 0;
  while (g + 1 < gr.n && o >= gr.first(g + 1)) ++g;
  const int co = gr.co(g), hc = co / 2, r = (o - gr.first(g)) % hc, hh = (o - gr.first(g)) / hc;
  uint8_t *slice = dst + slice_at(gr, F_in, g, ib >> 1, hh);
  const int kc = ib & 1;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    // panel and row: c = 0, 7 the real bins; c = 2b - 1 Wr, c = 2b Wi of bin b
    const int panel = c == 0 ? 0 : c == 7 ? 1 : 1 + (c + 1) / 2;
    const int rows = panel < 2 ? hc : co;
    const int row = panel < 2 || c % 2 == 0 ? r : hc + r;
    *reinterpret_cast<uint4 *>(slice + panel_at(panel, co) + (kc * rows + row) * 16) =
        make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]);
  }
}

struct DevCache {
  int clusters[2] = {};
};
std::mutex g_mu;
DevCache g_cache[64];

template <bool H>
int launch_wide(const void *x, const void *pack, void *y, int64_t T, int F_in, int F_out, cudaStream_t s) {
  auto kern = spectral8_wide_kernel<H>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
    return set_error(EQLIN_ERR_CUDA, "cudaGetDevice failed");
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int maxc = 0;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    int &n = g_cache[dev].clusters[H];
    if (!n) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
      if (e != cudaSuccess) return set_error(EQLIN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
      cfg.gridDim = dim3(2, 1, 1);
      cfg.dynamicSmemBytes = kSmemLimit;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess || n <= 0) {
        n = 0;
        return set_error(EQLIN_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
      }
    }
    maxc = n;
  }
  const Groups gr(F_out);
  const int co_big = gr.co(0), co_small = gr.co(gr.n - 1);
  CUtensorMap mx, mb, ms;
  int rc = tma_map_2d_bf16(&mx, x, (uint64_t)F_in * 8, (uint64_t)T, (uint64_t)F_in * 16, 64, kRows, true);
  if (rc) return rc;
  const uint64_t brows = (uint64_t)(slice_at(gr, F_in, gr.n - 1, F_in / 16, 0) / 512);
  rc = tma_map_2d_bf16(&mb, pack, 256, brows, 512, 256, (uint32_t)(slice_bytes(co_big) / 512), false);
  if (rc) return rc;
  rc = tma_map_2d_bf16(&ms, pack, 256, brows, 512, 256, (uint32_t)(slice_bytes(co_small) / 512), false);
  if (rc) return rc;
  WideArgs a;
  rc = fault_word_address(&a.fault);
  if (rc) return rc;
  a.y = y;
  a.epoch = next_launch_epoch();
  a.T = T;
  a.F_in = F_in;
  a.F_out = F_out;
  a.units = (int)((T + kTileTokens - 1) / kTileTokens) * gr.n;
  a.slot_bytes = kABytes + slice_bytes(co_big);
  a.nslots = (kSmemLimit - 1024 - kCtrl) / a.slot_bytes;
  if (a.nslots > kMaxSlots) a.nslots = kMaxSlots;
  // a round's pairs take whole tiles (a multiple of the groups)
  int npairs = maxc / gr.n * gr.n;
  if (npairs < 1) npairs = maxc;
  if (npairs > a.units) npairs = a.units;
  cfg.gridDim = dim3(2 * npairs, 1, 1);
  cfg.dynamicSmemBytes = 1024 + (size_t)a.nslots * a.slot_bytes + kCtrl;
  cfg.stream = s;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, mx, mb, ms, a);
  if (e != cudaSuccess) return set_error(EQLIN_ERR_CUDA, "wide tensor-core launch: %s", cudaGetErrorString(e));
  return check_launch("spectral8_wide_kernel");
}

}  // namespace

bool wide_tc_supported(int N, int F_in, int F_out, int dtype) {
  return (dtype == EQLIN_BF16 || dtype == EQLIN_F16) && N == 8 && F_in >= 16 && F_in % 16 == 0 && F_out >= 8 &&
         F_out % 8 == 0 && F_in <= (1 << 16) && F_out <= (1 << 16);
}

size_t wide_tc_bytes(int F_in, int F_out) {
  const Groups gr(F_out);
  return (size_t)slice_at(gr, F_in, gr.n - 1, F_in / 16, 0);
}

int launch_wide_tc_pack(const void *W, int F_in, int F_out, bool adjoint, int dtype, void *Ws, void *dst, cudaStream_t s) {
  const int64_t n = (int64_t)(Groups(F_out).blocks * kCoStep) * (F_in / 8);
  const unsigned grid = (unsigned)((n + 255) / 256);
  const uint4 *w = static_cast<const uint4 *>(W);
  float *ws = static_cast<float *>(Ws);
  uint8_t *d = static_cast<uint8_t *>(dst);
  if (dtype == EQLIN_F16)
    adjoint ? pack_wide_kernel<true, true><<<grid, 256, 0, s>>>(w, F_in, F_out, ws, d)
            : pack_wide_kernel<true, false><<<grid, 256, 0, s>>>(w, F_in, F_out, ws, d);
  else
    adjoint ? pack_wide_kernel<false, true><<<grid, 256, 0, s>>>(w, F_in, F_out, ws, d)
            : pack_wide_kernel<false, false><<<grid, 256, 0, s>>>(w, F_in, F_out, ws, d);
  return check_launch("wide tensor-core weight packing");
}

int launch_wide_tc(const void *x, const void *pack, void *y, int64_t T, int F_in, int F_out, int dtype,
                   cudaStream_t s) {
  if (T > (int64_t)0x7fff0000LL / Groups(F_out).n) return set_error(EQLIN_ERR_UNSUPPORTED, "T too large");
  return dtype == EQLIN_F16 ? launch_wide<true>(x, pack, y, T, F_in, F_out, s)
                            : launch_wide<false>(x, pack, y, T, F_in, F_out, s);
}

}  // namespace eqlin
