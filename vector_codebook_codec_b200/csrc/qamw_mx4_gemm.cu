// qamw_mx4_gemm.cu -- the product of two microscaled 4-bit matrices on the
// block-scaled tensor cores:  Y[t][m] = sum_j x[t][j] w[m][j].
//
// tcgen05.mma kind::mxf4 multiplies e2m1 elements with one e8m0 scale per 32
// of them and accumulates in fp32, 64 columns an instruction. A pipeline stage
// is 256 columns (128 bytes of codes per row, one swizzle atom) with its
// scales, which lie in the 128 x 4 tiles in which the tensor cores want them
// and are copied into tensor memory by the MMA thread (tcgen05.cp), in order
// with the MMAs that use them.
//
// Two kernels:
//  - up to 128 tokens: a CTA's tile is 128 weight rows (the tensor-memory
//    lanes) by NT tokens; the weights are all there is to read, so the columns
//    are split over a cluster until the SMs are busy, and the parts are added
//    in shared memory in the order of the ranks. The kernel alone (one after
//    another in a graph, other weights each time): 37 tokens x 13824 x 5120 12 us
//    (3.1 TB/s with its start and end), 128 tokens 13, 1 token x 4096 x 4096 6 us;
//  - more tokens: a pair of CTAs (cta_group::2) takes 256 tokens x 256 weight
//    rows, persistent. A token is a lane, so its outputs are contiguous. 4096
//    tokens x 11008 x 4096: 76 us (4.9 PFLOP/s), 4096 x 4096 x 16384: 105 us back to
//    back (5.3); a step's MMAs take 594 of 512 nominal cycles whether or not
//    anything is loaded, and the accumulator's drain 1.3 of 13 thousand cycles a
//    tile: two accumulators of 256 columns and the scales do not fit tensor memory
//    together (two of 192 would; not tried).
#include <algorithm>

#include "qamw_device.cuh"
#include "qamw_internal.h"
#include "qamw_tcgen05.cuh"

namespace qamw {
namespace {

constexpr int kBK = 256;          // columns per stage
constexpr int kRowBytes = 128;    // kBK / 2
constexpr int kSfTile = 512;      // bytes of a 128 x 4 scale tile
constexpr int kMaxStages = 8;
constexpr int kSfBufs = 4;        // scale buffers in tensor memory

struct MxGemmArgs {
  const uint8_t *w_scales, *x_scales;
  int64_t M, T, K, ldy;
  int64_t k_tiles;                // 128-column scale tiles of a row tile
  tc::TileWalk walk;              // pair kernel: token tiles x weight tiles
  void *Y;
  int out_bf16;
  int stages;
  int splits;                     // split kernel: CTAs of a cluster
  int steps_per_split;
  int after_quantize;             // x is still being written by the kernel before this one
  int32_t *status;
};

template <int CTAS>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else   // each CTA of the pair from its own shared memory into its own tensor memory
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// One stage: its scales into tensor memory (per 128 columns one scale tile of A
// and XB of B), then its MMAs of 64 columns; a scale tile's bytes 0-1 and 2-3
// (the scale ids) serve two of them. FULL: 256 columns, without a test.
// a, b, fa, fb: low descriptor words; sf: the stage's tensor-memory columns.
template <int CTAS, int XB, bool FULL>
__device__ __forceinline__ void stage(uint32_t d, uint32_t a, uint32_t b, uint32_t fa, uint32_t fb, uint32_t sf,
                                      uint32_t idesc, int left, bool fresh) {
  constexpr uint32_t kTile = kSfTile >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FULL || left > 128 * h) {
      cp_scales<CTAS>(sf + 4 * h, tc::desc(fa + kTile * h, tc::kDescScalesHi));
#pragma unroll
      for (int x = 0; x < XB; ++x)
        cp_scales<CTAS>(sf + 8 + 4 * (XB * h + x), tc::desc(fb + 2 * kTile * x + kTile * h, tc::kDescScalesHi));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (FULL || left > 64 * i)
      mma_mxf4<CTAS>(d, tc::desc(a + 2 * i, tc::kDescSw128Hi), tc::desc(b + 2 * i, tc::kDescSw128Hi),
                     idesc | ((uint32_t)(2 * (i & 1)) << 4) | ((uint32_t)(2 * (i & 1)) << 29), sf + 4 * (i >> 1),
                     sf + 8 + 4 * XB * (i >> 1), (!fresh || i != 0) ? 1u : 0u);
}
// e2m1 x e2m1 -> fp32, e8m0 scales, rows x cols
__host__ __device__ constexpr uint32_t idesc_of(int rows, int cols) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) | (1u << 23) | ((uint32_t)(rows >> 4) << 24);
}

// ---------------------------------------------------------------------------
// up to 128 tokens: 128 weight rows x NT tokens, columns split over a cluster
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 192;   // warp 0: loads, warp 1: MMA, warps 2-5: epilogue
template <int NT>
struct SplitTile {
  static constexpr int kA = 128 * kRowBytes, kB = NT * kRowBytes;
  static constexpr int kSf = 2 * kSfTile;                       // two scale tiles, of A and of B alike
  static constexpr int kStage = kA + kB + 2 * kSf;
  static constexpr int kCols = NT + kSfBufs * 16 <= 128 ? 128 : 256;
};

template <int NT>
__global__ void __launch_bounds__(kSplitThreads, 1)
    mx4_split_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MxGemmArgs g) {
  using L = SplitTile<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full;
  __shared__ uint32_t tmem_slot;
  __shared__ int fail_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  volatile int *fail = &fail_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = g.stages;
  uint8_t *sA = smem, *sB = smem + (size_t)S * L::kA, *sF = sB + (size_t)S * L::kB;
  const int rank = g.splits > 1 ? (int)tc::cta_rank() : 0;
  const int64_t mt = blockIdx.x / g.splits;
  const int all = (int)((g.K + kBK - 1) / kBK);
  const int k0 = rank * g.steps_per_split, k1 = min(k0 + g.steps_per_split, all);   // never empty

  auto sf_bytes = [&](int k) { return (uint32_t)(g.k_tiles - 2 * k >= 2 ? 2 * kSfTile : kSfTile); };
  auto load_w = [&](int k, uint32_t s) {
    if (tc::elect_one()) {
      mbar_arrive_expect_tx(&full[s], L::kA + L::kB + 2 * sf_bytes(k));
      tc::load_2d(sA + (size_t)s * L::kA, &wmap, k * kRowBytes, (int)(mt * 128), &full[s]);
      tc::load_bulk(sF + (size_t)s * 2 * L::kSf, g.w_scales + (mt * g.k_tiles + 2 * k) * kSfTile, sf_bytes(k),
                    &full[s]);
    }
  };
  const int n = k1 - k0, early = min(n, S);
  if (warp == 0) {
    if (lane == 0) {
      fail_flag = 0;
      for (int i = 0; i < S; ++i) {
        mbar_init(&full[i], 1);
        mbar_init(&empty[i], 1);
      }
      mbar_init(&acc_full, 1);
      tc::mbar_init_fence();
    }
    __syncwarp();
    // the weights of the first stages are on their way while the CTA sets up and x is still being coded
    for (int i = 0; i < early; ++i) load_w(k0 + i, i);
  }
  if (warp == 1) tc::alloc(&tmem_slot, L::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  uint32_t bad = 0;
  // by every thread, before any role's bounded waits begin: they then cover this kernel's own time only
  if (g.after_quantize) tc::griddep_wait();

  if (warp == 0) {
    auto load_x = [&](int k, uint32_t s) {
      if (tc::elect_one()) {
        tc::load_2d(sB + (size_t)s * L::kB, &xmap, k * kRowBytes, 0, &full[s]);
        tc::load_bulk(sF + (size_t)s * 2 * L::kSf + L::kSf, g.x_scales + 2 * (int64_t)k * kSfTile, sf_bytes(k),
                      &full[s]);
      }
    };
    for (int i = 0; i < early; ++i) load_x(k0 + i, i);
    int it = early;
    for (tc::Ring r; it < n; ++it, r.next(S)) {
      if (!tc::wait(&empty[r.s], r.phase, fail)) break;
      load_w(k0 + it, r.s);
      load_x(k0 + it, r.s);
    }
    if (*fail) {   // leave no copy in flight behind
      for (int i = max(it - S, 0); i < it; ++i) mbar_wait(&full[i % S], (i / S) & 1u, tc::kWaitTries);
      bad |= QAMW_STATUS_TIMEOUT;
    }
  } else if (warp == 1) {
    const uint32_t a = tc::desc_lo(sA), b = tc::desc_lo(sB), f = tc::desc_lo(sF);
    tc::Ring r;
    for (int k = k0; k < k1; ++k, r.next(S)) {
      if (!tc::wait(&full[r.s], r.phase, fail)) { bad |= QAMW_STATUS_TIMEOUT; break; }
      tc::fence_after();
      if (tc::elect_one()) {
        const uint32_t sa = a + r.s * (L::kA >> 4), sb = b + r.s * (L::kB >> 4), fs = f + r.s * (2 * L::kSf >> 4);
        const uint32_t sf = tmem + NT + ((k - k0) % kSfBufs) * 16;
        const int left = (int)g.K - k * kBK;
        if (left >= kBK)
          stage<1, 1, true>(tmem, sa, sb, fs, fs + (L::kSf >> 4), sf, idesc_of(128, NT), left, k == k0);
        else
          stage<1, 1, false>(tmem, sa, sb, fs, fs + (L::kSf >> 4), sf, idesc_of(128, NT), left, k == k0);
        tc::commit(&empty[r.s]);
      }
      __syncwarp();
    }
    if (tc::elect_one()) tc::commit(&acc_full);   // after a failure too: the MMAs in flight are waited for below
  }
  __syncwarp();
  // every warp: the MMAs (hence all loads) are done
  if (!tc::wait_warp(&acc_full, 0u, fail)) bad |= QAMW_STATUS_TIMEOUT;
  tc::fence_after();
  const int wq = warp & 3;
  const int64_t m = mt * 128 + 32 * wq + lane;
  auto put = [&](int64_t t, float v) {
    if (m < g.M && t < g.T) {
      if (g.out_bf16) static_cast<__nv_bfloat16 *>(g.Y)[t * g.ldy + m] = __float2bfloat16_rn(v);
      else static_cast<float *>(g.Y)[t * g.ldy + m] = v;
    }
  };
  // Tensor memory is given back before the CTAs of a cluster wait for one
  // another: a CTA of another kernel (or cluster) that waits for it on this SM
  // may be the one that a holder elsewhere waits for.
  float *part = reinterpret_cast<float *>(smem);   // [NT][128], in the memory of the stages
  if (warp >= 2 && g.splits == 1) {
    auto write = [&](auto *y, auto rounded) {       // one type for the whole tile
      y += m;
      for (int c0 = 0; c0 < NT && c0 < g.T; c0 += 16, y += 16 * g.ldy) {
        float v[16];
        tc::ld16(tmem + (uint32_t)c0 + ((uint32_t)(32 * wq) << 16), v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (m < g.M && c0 + j < g.T) y[j * g.ldy] = rounded(v[j]);
      }
    };
    if (g.out_bf16) write(static_cast<__nv_bfloat16 *>(g.Y), [](float v) { return __float2bfloat16_rn(v); });
    else write(static_cast<float *>(g.Y), [](float v) { return v; });
  } else if (warp >= 2) {
    for (int c0 = 0; c0 < NT && c0 < g.T; c0 += 16) {
      float v[16];
      tc::ld16(tmem + (uint32_t)c0 + ((uint32_t)(32 * wq) << 16), v);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + 32 * wq + lane] = v[j];
    }
  }
  tc::fence_before();
  __syncthreads();
  if (g.splits > 1) tc::cluster_arrive();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, L::kCols);
    __syncwarp();
  }
  if (g.splits > 1) {
    tc::cluster_wait();
    if (warp >= 2) {
      // rank r adds and writes tokens r, r + splits, ...: four tokens' parts of up to 8 ranks in flight
      // together, added in the order of the ranks
      for (int64_t t0 = rank; t0 < g.T; t0 += 4 * g.splits) {
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t t = t0 + i * g.splits;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            v[i][r] = r < g.splits && t < g.T ? tc::ld_cluster(tc::address_in(&part[t * 128 + 32 * wq + lane], r)) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float sum = v[i][0];
#pragma unroll
          for (int r = 1; r < 8; ++r) sum += v[i][r];   // a rank that is not there adds 0
          put(t0 + i * g.splits, sum);
        }
      }
    }
    __syncwarp();
    tc::cluster_sync();   // no CTA leaves while its part is read
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) status_or(g.status, bad);
}

// ---------------------------------------------------------------------------
// more than 128 tokens: 256 tokens x 256 weight rows for a pair of CTAs
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 320;    // warp 0: loads, warp 1: MMA, warps 2-9: epilogue
constexpr int kPairA = 128 * kRowBytes, kPairB = 128 * kRowBytes;   // each CTA loads half of both operands
constexpr int kPairSfA = 2 * kSfTile, kPairSfB = 4 * kSfTile;       // but the scales of all 256 weight rows
constexpr int kPairStage = kPairA + kPairB + kPairSfA + kPairSfB;
constexpr int kPairSfCols = 24;                                     // tensor-memory columns of a stage's scales

__global__ void __launch_bounds__(kPairThreads, 1)
    mx4_pair_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                    const __grid_constant__ CUtensorMap wsmap, const __grid_constant__ CUtensorMap xsmap,
                    MxGemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty, drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int fail_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  volatile int *fail = &fail_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cta_rank();
  const int S = g.stages;
  uint8_t *sA = smem, *sB = smem + (size_t)S * kPairA, *sF = sB + (size_t)S * kPairB;

  if (threadIdx.x == 0) {
    fail_flag = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&acc_empty, 16);         // 8 epilogue warps of each CTA
    mbar_init(&drained, 1);
    tc::mbar_init_fence();
  }
  if (warp == 1) tc::alloc_pair(&tmem_slot, 512);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();   // both CTAs' barriers exist before either is signalled
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  const int64_t n_tiles = g.walk.n_r * g.walk.n_c, step = gridDim.x / 2, first = blockIdx.x / 2;
  const int n_k = (int)((g.K + kBK - 1) / kBK);
  uint32_t bad = 0;
  if (g.after_quantize) tc::griddep_wait();   // by every thread, before any role's bounded waits begin

  if (warp == 0) {
    uint32_t it = 0;
    tc::Ring r;
    bool ok = true;
    for (int64_t tile = first; tile < n_tiles && ok; tile += step) {
      int64_t rt, ct;
      g.walk.at(tile, rt, ct);
      const int x0 = (int)(rt * 256 + rank * 128), w0 = (int)(ct * 256 + rank * 128);
      // first scale tiles of the rows; a tile past the last row is filled with zeros, and one past
      // the end of K (the next row's first) is not used
      const int xr = (int)((2 * rt + rank) * g.k_tiles), wr = (int)(2 * ct * g.k_tiles), kt = (int)g.k_tiles;
      for (int k = 0; k < n_k; ++k, ++it, r.next(S)) {
        if (!tc::wait(&empty[r.s], r.phase ^ 1u, fail)) { ok = false; break; }
        if (tc::elect_one()) {
          // the leader's barrier counts the bytes of both CTAs, and the leader alone announces them (an
          // announcement of each CTA at the other's barrier cost more than the stage's MMAs)
          if (rank == 0) mbar_arrive_expect_tx(&full[r.s], 2 * kPairStage);
          const uint32_t lb = tc::address_in(&full[r.s], 0);
          tc::load_2d_pair(sA + (size_t)r.s * kPairA, &xmap, k * kRowBytes, x0, lb);
          tc::load_2d_pair(sB + (size_t)r.s * kPairB, &wmap, k * kRowBytes, w0, lb);
          uint8_t *f = sF + (size_t)r.s * (kPairSfA + kPairSfB);
          tc::load_2d_pair(f, &xsmap, 0, xr + 2 * k, lb);
          tc::load_2d_pair(f + kPairSfA, &wsmap, 0, wr + 2 * k, lb);
          tc::load_2d_pair(f + kPairSfA + 2 * kSfTile, &wsmap, 0, wr + kt + 2 * k, lb);
        }
        __syncwarp();
      }
    }
    if (*fail) {   // leave no copy in flight behind (the leader's barriers count both CTAs')
      if (rank == 0) {
        const uint32_t from = it > (uint32_t)S ? it - S : 0;
        for (uint32_t i = from; i < it; ++i) mbar_wait(&full[i % S], (i / S) & 1u, tc::kWaitTries);
      }
      bad |= QAMW_STATUS_TIMEOUT;
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t a = tc::desc_lo(sA), b = tc::desc_lo(sB), f = tc::desc_lo(sF);
      uint32_t sfb = 0, seg = 0;
      tc::Ring r;
      bool ok = true;
      for (int64_t tile = first; tile < n_tiles && ok; tile += step, ++seg) {
        if (!tc::wait(&acc_empty, (seg & 1u) ^ 1u, fail)) break;
        tc::fence_after();
        for (int k = 0; k < n_k; ++k, r.next(S), sfb = (sfb + 1) % kSfBufs) {
          if (!tc::wait(&full[r.s], r.phase, fail)) { ok = false; break; }
          tc::fence_after();
          if (tc::elect_one()) {
            const uint32_t sa = a + r.s * (kPairA >> 4), sb = b + r.s * (kPairB >> 4);
            const uint32_t fs = f + r.s * ((kPairSfA + kPairSfB) >> 4), sf = tmem + 256 + sfb * kPairSfCols;
            const int left = (int)g.K - k * kBK;
            if (left >= kBK)
              stage<2, 2, true>(tmem, sa, sb, fs, fs + (kPairSfA >> 4), sf, idesc_of(256, 256), left, k == 0);
            else
              stage<2, 2, false>(tmem, sa, sb, fs, fs + (kPairSfA >> 4), sf, idesc_of(256, 256), left, k == 0);
            tc::commit_pair(&empty[r.s]);
            if (k == n_k - 1) tc::commit_pair(&acc_full);
          }
          __syncwarp();
        }
      }
      if (*fail) {
        if (tc::elect_one()) tc::commit_pair(&drained);
        mbar_wait(&drained, 0u, tc::kWaitTries);
        bad |= QAMW_STATUS_TIMEOUT;
      }
    }
  } else {
    // a warp takes 32 tokens x 128 outputs: the accumulators are read into
    // registers at once and handed back, so that the next tile's MMAs run while
    // the outputs are written
    const int wq = warp & 3, half = (warp - 2) >> 2;
    uint32_t seg = 0;
    for (int64_t tile = first; tile < n_tiles; tile += step, ++seg) {
      int64_t rt, ct;
      g.walk.at(tile, rt, ct);
      if (!tc::wait_warp(&acc_full, seg & 1u, fail)) { bad |= QAMW_STATUS_TIMEOUT; break; }
      tc::fence_after();
      float v[128];
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::ld32_async(tmem + 128 * half + 32 * c + ((uint32_t)(32 * wq) << 16), v + 32 * c);
      tc::ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) tc::tie32(v + 32 * c);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive_cluster(tc::address_in(&acc_empty, 0));
      const int64_t t = rt * 256 + rank * 128 + 32 * wq + lane, m = ct * 256 + 128 * half;
      if (t < g.T) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t at = t * g.ldy + m + 32 * c, n = g.M - (m + 32 * c);
          if (n > 0) {
            if (g.out_bf16) tc::store_row32(static_cast<__nv_bfloat16 *>(g.Y) + at, n < 32 ? (int)n : 32, v + 32 * c);
            else tc::store_row32(static_cast<float *>(g.Y) + at, n < 32 ? (int)n : 32, v + 32 * c);
          }
        }
      }
    }
  }

  __syncwarp();
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();   // no CTA leaves while the pair's MMAs, copies or arrivals may reach it
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc_pair(tmem, 512);
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) status_or(g.status, bad);
}

bool make_map(CUtensorMap *m, const uint8_t *codes, int64_t rows, int64_t K, int box_rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
  cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as rows of 128 words, loaded two at a time: a tensor copy, since
// only that may count its bytes at the pair's other CTA.
bool make_scale_map(CUtensorMap *m, const uint8_t *scales, int64_t row_tiles, int64_t k_tiles) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {kSfTile / 4, (cuuint64_t)(row_tiles * k_tiles)};
  cuuint64_t strides[1] = {kSfTile};
  cuuint32_t box[2] = {kSfTile / 4, 2};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t *>(scales), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Kernel, typename... Args>
cudaError_t launch(Kernel kernel, int grid, int threads, size_t smem, int cluster, bool dependent, cudaStream_t s,
                   const Args &...args) {
  const cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NT>
cudaError_t run_split(const Mx4MatmulArgs &a, MxGemmArgs g, int smem_max, cudaStream_t s) {
  using L = SplitTile<NT>;
  CUtensorMap wmap, xmap;
  if (!make_map(&wmap, a.w_codes, a.M, a.K, 128) || !make_map(&xmap, a.x_codes, a.T, a.K, NT))
    return cudaErrorInvalidValue;
  // Splits: the power of two that minimises waves x (steps of a CTA + 4, the
  // steps' worth of a CTA's start and end). One CTA per SM with all its memory:
  // two with half of it, and twice the splits, were slower (whole calls then: 37
  // tokens x 13824 x 5120 16 us, in halves 22; 128 tokens 18 and 37, most of it for
  // adding the parts).
  const int64_t tiles = (a.M + 127) / 128, steps = (a.K + kBK - 1) / kBK;
  int64_t best = INT64_MAX;
  for (int sp = 1; sp <= 8 && sp <= steps; sp *= 2) {
    const int64_t per = (steps + sp - 1) / sp;
    if ((steps + per - 1) / per != sp) continue;       // a rank without work
    const int64_t cost = ((tiles * sp + sm_count() - 1) / sm_count()) * (per + 4);
    if (cost < best) best = cost, g.splits = sp, g.steps_per_split = (int)per;
  }
  g.stages = (int)std::min<int64_t>(std::min<int64_t>(kMaxStages, (smem_max - 2048) / L::kStage), g.steps_per_split);
  // the parts (NT x 128 fp32) lie in the memory of the stages
  const size_t bytes = std::max<size_t>((size_t)g.stages * L::kStage, g.splits > 1 ? (size_t)NT * 128 * 4 : 0);
  return launch(mx4_split_kernel<NT>, (int)(tiles * g.splits), kSplitThreads, 1024 + bytes, g.splits,
                a.after_quantize, s, wmap, xmap, g);
}

cudaError_t run_pair(const Mx4MatmulArgs &a, MxGemmArgs g, int smem_max, cudaStream_t s) {
  CUtensorMap wmap, xmap, wsmap, xsmap;
  if (!make_map(&wmap, a.w_codes, a.M, a.K, 128) || !make_map(&xmap, a.x_codes, a.T, a.K, 128) ||
      !make_scale_map(&wsmap, a.w_scales, (a.M + 127) / 128, g.k_tiles) ||
      !make_scale_map(&xsmap, a.x_scales, (a.T + 127) / 128, g.k_tiles))
    return cudaErrorInvalidValue;
  g.walk = tc::TileWalk{(a.T + 255) / 256, (a.M + 255) / 256, 16};
  g.stages = (int)std::min<int64_t>(kMaxStages, (smem_max - 2048) / kPairStage);
  const int64_t pairs = std::min<int64_t>(sm_count() / 2, g.walk.n_r * g.walk.n_c);
  return launch(mx4_pair_kernel, (int)(2 * pairs), kPairThreads, 1024 + (size_t)g.stages * kPairStage, 2,
                a.after_quantize, s, wmap, xmap, wsmap, xsmap, g);
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs &a, cudaStream_t s) {
  int dev = 0, smem_max = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  MxGemmArgs g = {};
  g.w_scales = a.w_scales;
  g.x_scales = a.x_scales;
  g.M = a.M;
  g.T = a.T;
  g.K = a.K;
  g.ldy = a.ldy;
  g.k_tiles = (a.K + 127) / 128;
  g.Y = a.Y;
  g.out_bf16 = a.out_t == QAMW_BF16;
  g.after_quantize = a.after_quantize;
  g.status = a.status;
  if (a.T <= 16) return run_split<16>(a, g, smem_max, s);
  if (a.T <= 32) return run_split<32>(a, g, smem_max, s);
  if (a.T <= 64) return run_split<64>(a, g, smem_max, s);
  if (a.T <= 128) return run_split<128>(a, g, smem_max, s);
  return run_pair(a, g, smem_max, s);
}

}  // namespace qamw
