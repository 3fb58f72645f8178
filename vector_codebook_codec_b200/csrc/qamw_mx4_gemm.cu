// qamw_mx4_gemm.cu -- the product of two microscaled 4-bit matrices on the
// block-scaled tensor cores:  Y[t][m] = sum_j x[t][j] w[m][j].
//
// tcgen05.mma kind::mxf4 multiplies e2m1 elements with one e8m0 scale per 32
// of them and accumulates in fp32, 64 columns an instruction. A tile is 128
// weight rows (the tensor-memory lanes) by NT tokens; a pipeline stage is 256
// columns (128 bytes of codes per row, one swizzle atom) with its scales. The
// scales arrive in the 128 x 4 tiles in which the tensor cores want them and
// are copied into tensor memory by the MMA thread (tcgen05.cp), in order with
// the MMAs that use them.
#include <algorithm>

#include "qamw_device.cuh"
#include "qamw_internal.h"
#include "qamw_tcgen05.cuh"

namespace qamw {
namespace {

constexpr int kBM = 128;          // weight rows per tile
constexpr int kBK = 256;          // columns per stage
constexpr int kRowBytes = 128;    // kBK / 2
constexpr int kThreads = 192;     // warp 0: loads, warp 1: MMA, warps 2-5: epilogue
constexpr int kMaxStages = 8;
constexpr int kSfBufs = 4;        // scale buffers in tensor memory

struct MxGemmArgs {
  const uint8_t *w_scales, *x_scales;
  int64_t M, T, K, ldy;
  int64_t k_tiles;                // 128-column scale tiles of a row tile
  int64_t x_row_tiles;            // 128-row scale tiles of x
  int64_t n_m, n_t;               // tiles
  void *Y;
  int out_bf16;
  int stages;
  int32_t *status;
};

template <int NT>
struct MxTile {
  static constexpr int kXBlocks = (NT + 127) / 128;             // 128-token scale tiles
  static constexpr int kA = kBM * kRowBytes;                    // bytes
  static constexpr int kB = (NT < 8 ? 8 : NT) * kRowBytes;
  static constexpr int kSfA = 1024, kSfB = 1024 * kXBlocks;     // two 512-byte tiles per 128 rows
  static constexpr int kStage = kA + kB + kSfA + kSfB;
  static constexpr int kAccs = NT <= 128 ? 2 : 1;
  static constexpr int kAccCols = NT;
  static constexpr int kSfCols = 8 + 8 * kXBlocks;              // per buffer
  static constexpr int kNeed = kAccs * kAccCols + kSfBufs * kSfCols;
  static constexpr int kCols = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
};

__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap, MxGemmArgs g) {
  using L = MxTile<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int fail_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  volatile int *fail = &fail_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = g.stages;
  // stage s: all A tiles, then all B tiles, then the scales (A and B stay 1024-byte aligned)
  uint8_t *sA = smem, *sB = smem + (size_t)S * L::kA, *sF = sB + (size_t)S * L::kB;

  if (threadIdx.x == 0) {
    fail_flag = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(&drained, 1);
    tc::mbar_init_fence();
  }
  if (warp == 1) tc::alloc(&tmem_slot, L::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_slot;
  const int64_t n_tiles = g.n_m * g.n_t;
  const int n_k = (int)((g.K + kBK - 1) / kBK);
  uint32_t bad = 0;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
        const int64_t mt = tile % g.n_m, tt = tile / g.n_m;
        const uint8_t *sfw = g.w_scales + mt * g.k_tiles * 512;
        for (int k = 0; k < n_k; ++k, ++it) {
          const uint32_t s = it % S;
          if (!tc::wait(&empty[s], ((it / S) & 1u) ^ 1u, fail)) { ok = false; break; }
          // 128-column scale tiles of this stage: two, or one at the end of K
          const int64_t kt = 2 * (int64_t)k;
          const uint32_t sf_bytes = g.k_tiles - kt >= 2 ? 1024u : 512u;
          uint32_t xb = 0;
#pragma unroll
          for (int b = 0; b < L::kXBlocks; ++b)
            if (tt * NT / 128 + b < g.x_row_tiles) ++xb;
          mbar_arrive_expect_tx(&full[s], L::kA + L::kB + sf_bytes * (1 + xb));
          tc::load_2d(sA + (size_t)s * L::kA, &wmap, k * kRowBytes, (int)(mt * kBM), &full[s]);
          tc::load_2d(sB + (size_t)s * L::kB, &xmap, k * kRowBytes, (int)(tt * NT), &full[s]);
          uint8_t *f = sF + (size_t)s * (L::kSfA + L::kSfB);
          tc::load_bulk(f, sfw + kt * 512, sf_bytes, &full[s]);
          for (uint32_t b = 0; b < xb; ++b)
            tc::load_bulk(f + L::kSfA + 1024 * b,
                          g.x_scales + ((tt * NT / 128 + b) * g.k_tiles + kt) * 512, sf_bytes, &full[s]);
        }
      }
      if (*fail) {   // leave no copy in flight behind
        const uint32_t first = it > (uint32_t)S ? it - S : 0;
        for (uint32_t i = first; i < it; ++i) mbar_wait(&full[i % S], (i / S) & 1u, tc::kWaitTries);
        bad |= QAMW_STATUS_TIMEOUT;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // e2m1 x e2m1 -> fp32, e8m0 scales, 128 x NT
      constexpr uint32_t kIdesc = (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) | (1u << 23) | (8u << 24);
      uint32_t it = 0, seg = 0;
      bool ok = true;
      for (int64_t tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x, ++seg) {
        const uint32_t buf = seg % L::kAccs;
        if (!tc::wait(&acc_empty[buf], ((seg / L::kAccs) & 1u) ^ 1u, fail)) break;
        tc::fence_after();
        const uint32_t d = tmem + buf * L::kAccCols;
        for (int k = 0; k < n_k; ++k, ++it) {
          const uint32_t s = it % S;
          if (!tc::wait(&full[s], (it / S) & 1u, fail)) { ok = false; break; }
          tc::fence_after();
          const uint32_t a = smem_u32(sA + (size_t)s * L::kA), b = smem_u32(sB + (size_t)s * L::kB);
          const uint32_t f = smem_u32(sF + (size_t)s * (L::kSfA + L::kSfB));
          const uint32_t sfa = tmem + L::kAccs * L::kAccCols + (it % kSfBufs) * L::kSfCols, sfb = sfa + 8;
          const int left = (int)(g.K - (int64_t)k * kBK);     // columns from here to the end
          const int n_mma = left >= kBK ? 4 : (left + 63) / 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) {                       // 128 columns: one scale tile, two MMAs
            if (2 * h < n_mma) {
              cp_scales(sfa + 4 * h, tc::desc_scales(f + 512 * h));
#pragma unroll
              for (int x = 0; x < L::kXBlocks; ++x)
                cp_scales(sfb + 4 * (L::kXBlocks * h + x), tc::desc_scales(f + L::kSfA + 1024 * x + 512 * h));
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int i = 2 * h + j;
                if (i < n_mma)
                  // scales 2j and 2j + 1 of each row's four: the scale ids of the descriptor
                  mma_mxf4(d, tc::desc_k_sw128(a + 32 * i), tc::desc_k_sw128(b + 32 * i),
                           kIdesc | ((uint32_t)(2 * j) << 4) | ((uint32_t)(2 * j) << 29), sfa + 4 * h,
                           sfb + 4 * L::kXBlocks * h, (k | i) != 0);
              }
            }
          }
          tc::commit(&empty[s]);
        }
        if (ok) tc::commit(&acc_full[buf]);
      }
      if (*fail) {
        tc::commit(&drained);
        mbar_wait(&drained, 0u, tc::kWaitTries);
        bad |= QAMW_STATUS_TIMEOUT;
      }
    }
  } else {
    const int wq = warp & 3;
    uint32_t seg = 0;
    for (int64_t tile = blockIdx.x; tile < n_tiles; tile += gridDim.x, ++seg) {
      const int64_t mt = tile % g.n_m, tt = tile / g.n_m;
      const uint32_t buf = seg % L::kAccs;
      if (!tc::wait(&acc_full[buf], (seg / L::kAccs) & 1u, fail)) { bad |= QAMW_STATUS_TIMEOUT; break; }
      __syncwarp();
      tc::fence_after();
      const int64_t m = mt * kBM + 32 * wq + lane;
      const uint32_t taddr = tmem + buf * L::kAccCols + ((uint32_t)(32 * wq) << 16);
      for (int c0 = 0; c0 < NT; c0 += 16) {
        float v[16];
        tc::ld16(taddr + (uint32_t)c0, v);
        const int64_t t0 = tt * NT + c0;
        if (m < g.M) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if (t0 + j < g.T) {
              if (g.out_bf16) static_cast<__nv_bfloat16 *>(g.Y)[(t0 + j) * g.ldy + m] = __float2bfloat16_rn(v[j]);
              else static_cast<float *>(g.Y)[(t0 + j) * g.ldy + m] = v[j];
            }
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
    }
  }

  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tmem, L::kCols);
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) status_or(g.status, bad);
}

template <int NT>
cudaError_t run(const Mx4MatmulArgs &a, cudaStream_t s) {
  using L = MxTile<NT>;
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  int dev = 0, smem_max = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  CUtensorMap wmap, xmap;
  auto make = [&](CUtensorMap *m, const uint8_t *codes, int64_t rows, int box_rows) {
    cuuint64_t dims[2] = {(cuuint64_t)(a.K / 2), (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(a.K / 2)};
    cuuint32_t box[2] = {(cuuint32_t)kRowBytes, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!make(&wmap, a.w_codes, a.M, kBM) || !make(&xmap, a.x_codes, a.T, NT)) return cudaErrorInvalidValue;
  MxGemmArgs g;
  g.w_scales = a.w_scales;
  g.x_scales = a.x_scales;
  g.M = a.M;
  g.T = a.T;
  g.K = a.K;
  g.ldy = a.ldy;
  g.k_tiles = (a.K + 127) / 128;
  g.x_row_tiles = (a.T + 127) / 128;
  g.n_m = (a.M + kBM - 1) / kBM;
  g.n_t = (a.T + NT - 1) / NT;
  g.Y = a.Y;
  g.out_bf16 = a.out_t == QAMW_BF16;
  g.status = a.status;
  g.stages = (int)std::min<int64_t>(kMaxStages, (smem_max - 2048) / L::kStage);
  const size_t smem = 1024 + (size_t)g.stages * L::kStage;
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void *>(mx4_gemm_kernel<NT>), smem)) != cudaSuccess) return e;
  const int64_t grid = std::min<int64_t>(sm_count(), g.n_m * g.n_t);
  mx4_gemm_kernel<NT><<<(unsigned)grid, kThreads, smem, s>>>(wmap, xmap, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4MatmulArgs &a, cudaStream_t s) {
  if (a.T <= 16) return run<16>(a, s);
  if (a.T <= 32) return run<32>(a, s);
  if (a.T <= 64) return run<64>(a, s);
  if (a.T <= 128) return run<128>(a, s);
  return run<256>(a, s);
}

}  // namespace qamw
