// qamw_cross_entropy.cu -- softmax cross entropy of a model's head without
// keeping the logits, and its gradient, a piece of the vocabulary at a time.
//
//   l_tv = sum_j X_tj W_vj;  lse_t = log sum_v exp l_tv;  loss_t = lse_t - l_t,target(t)
//   G_tv = g_t (exp(l_tv - lse_t) - [v = target(t)]);  dX = G W;  dW = G^T X
//
// G is kept as G / max|g|, and the fp32 sums are multiplied by max|g|: with the
// mean's equal g_t the entries near -1, which carry most of both gradients, are
// then all but exact in bf16 instead of all being off by the rounding of g
// (relative error of dX against 64 bits at 4096 tokens x 65536: 3.6e-3 -> the
// 1.7e-3 of the output's own rounding).
//
// All three products run through one tcgen05 kernel (bf16 operands, fp32
// accumulation in tensor memory) whose epilogue consumes the accumulators
// where they are: the forward pass reduces 128 logits of a token to their
// maximum and sum of exponentials (8 bytes leave the SM instead of 512), the
// backward pass turns them into G. G of one piece is the only matrix of
// that size that exists, rounded to bf16 once (2^-8 relative at most; two terms
// for few tokens, see kTwoTerms): bf16 is the operand type that W and X have,
// and one tcgen05 product takes one type.
//
// A tile is 256 rows x 256 columns for a pair of CTAs (cta_group::2, 128
// accumulator rows each; every CTA loads half of both operands), or 128 x 256
// for one CTA (single_cta below). 8 epilogue warps work on one accumulator while
// the MMAs fill the other.
//
// Bound by power for large products: 4096 tokens x 32000 x 4096 forward takes
// 0.64 ms in a run of 20 calls (1.68 PFLOP/s) and 0.78 ms back to back, the
// gradient of 4096 x 65536 x 4096 4.2 and 4.9 ms (1.57 and 1.35 PFLOP/s over its
// three products). For few tokens by the read of W: 16 x 32000 x 2048 takes 30 us,
// 4.4 TB/s with its start and finish, 16 x 32000 x 8192 88 us, 5.9 TB/s.
//
// The tensor cores add in fp32 and cut off what lies below the sum's last bit, so
// logits are off by about K / 16 x 2^-24 of their size: lse of 4096 columns by
// 7.6e-7 of itself (with rounding 8e-8), a loss by some 1e-5.
#include <algorithm>

#include "qamw_device.cuh"
#include "qamw_internal.h"
#include "qamw_tcgen05.cuh"

namespace qamw {
namespace {

constexpr int kBN = 256;          // columns per tile
constexpr int kBK = 64;           // contraction per stage: 128 bytes of bf16
constexpr int kThreads = 320;     // warp 0: loads, warp 1: MMA, warps 2-9: epilogue
constexpr int kHalf = 128;        // columns of a tile that an epilogue warp takes
constexpr int kBox = 64 * 128;    // bytes of a 64 x 64 box
constexpr int kMaxStages = 8;
constexpr int kShortDepth = 256;  // contraction up to which bf16 outputs leave by TMA stores (see run())
constexpr int kGroupRows = 16;    // row tiles walked together (their operand stays in L2)

enum Epilogue { kStats = 0, kGrad = 1, kGradTwo = 2, kStore = 3, kSlot = 4 };   // kGradTwo: kGrad, two terms

struct CeArgs {
  int64_t rows, cols, depth;      // of the product: D[rows][cols], contraction over depth
  int64_t n_r, n_c;               // tiles
  int splits;                     // contraction split (kSlot only)
  int64_t steps_per_split;
  int stages;
  int a_bytes;                    // of a stage's row operand: rows x 128
  int32_t *status;
  // kStats, kGrad, kGradTwo: rows are tokens, columns the vocabulary entries v0 ..
  const int64_t *targets;         // [T]
  int64_t v0, V, ignore;
  float2 *partials;               // kStats: [half tiles of the whole vocabulary][T] (maximum, sum relative to it)
  float *target_logit;            // kStats: [T]
  const float *lse, *grad;        // kGrad, kGradTwo: [T]
  const float *factor;            // kGrad, kGradTwo: of G (divided out); kStore: of D
  __nv_bfloat16 *out;             // kGrad: G, kGradTwo: its terms below one another, kStore: D
  int64_t ldo;
  int tma_out;                    // they leave by TMA stores
  float *slots;                   // kSlot: [splits][rows][cols] fp32
  int add;                        // kSlot: add to the slots instead of writing them
};

template <int CTAS>
struct CeTile {
  static constexpr int kRows = 128 * CTAS;                  // rows per tile
  static constexpr int kColsHere = kBN / CTAS;              // operand columns that one CTA loads
  static constexpr int kB = kColsHere * 128;                // bytes per stage
};

// Operands whose rows (or columns) of the product are contiguous: a 64 x 64 box
// holds 64 contraction rows of 128 bytes; 8-row atoms are 1024 bytes apart
// along the contraction (as in the other layout), boxes 8192 bytes along the
// rows (the leading offset). 16 contraction steps are 2048 bytes, or 32 bytes
// where the contraction is contiguous.
template <bool MN>
__device__ __forceinline__ uint32_t operand_lo(const void *p) {
  return tc::desc_lo(p, MN ? kBox >> 4 : 1);
}

template <int CTAS>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5, %5, %5, %5, %5}, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(0u)
        : "memory");
}
template <int CTAS>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (CTAS == 1) tc::commit(bar);
  else tc::commit_pair(bar);
}
template <int CTAS>
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar,
                                         uint32_t leader_bar) {
  if constexpr (CTAS == 1) tc::load_2d(dst, map, x, y, bar);
  else tc::load_2d_pair(dst, map, x, y, leader_bar);
}

struct Unit {                     // one tile (and contraction range) of the walk
  int64_t rt, ct;
  int split;
  int64_t k0, k1;                 // contraction steps
};
__device__ __forceinline__ Unit unit_of(const CeArgs &g, int64_t u) {
  Unit r;
  const int64_t tiles = g.n_r * g.n_c;
  r.split = (int)(u / tiles);
  const int64_t t = u - r.split * tiles;
  tc::TileWalk{g.n_r, g.n_c, kGroupRows}.at(t, r.rt, r.ct);
  const int64_t all = (g.depth + kBK - 1) / kBK;
  r.k0 = r.split * g.steps_per_split;
  r.k1 = r.k0 + g.steps_per_split < all ? r.k0 + g.steps_per_split : all;
  if (r.k0 > all) r.k0 = all;
  return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// log2 of exp(a) / exp(ref) and of exp(b) / exp(ref)
__device__ __forceinline__ float2 log2_ratio(float a, float b, float ref) {
  return mul2(add2(make_float2(a, b), make_float2(-ref, -ref)), make_float2(kLog2e, kLog2e));
}

// A_MN / B_MN: the operand lies [contraction][rows or columns] in memory.
template <int CTAS, bool A_MN, bool B_MN, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                   const __grid_constant__ CUtensorMap omap, CeArgs g) {
  using L = CeTile<CTAS>;
  constexpr bool kIsGrad = EPI == kGrad || EPI == kGradTwo;
  tc::griddep_launch_dependents();   // the next kernel may set up; it waits for this one before it reads or writes
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ int fail_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  volatile int *fail = &fail_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CTAS == 1 ? 0u : tc::cta_rank();
  const int S = g.stages;
  uint8_t *sA = smem, *sB = smem + S * g.a_bytes;

  if (threadIdx.x == 0) {
    fail_flag = 0;
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8 * CTAS);
    }
    mbar_init(&drained, 1);
    tc::mbar_init_fence();
  }
  if (warp == 1) {
    if constexpr (CTAS == 1) tc::alloc(&tmem_slot, 512);
    else tc::alloc_pair(&tmem_slot, 512);
  }
  tc::fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) tc::cluster_sync();   // both CTAs' barriers exist before either is signalled
  tc::fence_after();
  tc::griddep_wait();
  const uint32_t tmem = tmem_slot;
  const int64_t n_units = g.n_r * g.n_c * g.splits, step = gridDim.x / CTAS, first = blockIdx.x / CTAS;
  uint32_t bad = 0;

  if (warp == 0) {
    uint32_t it = 0;
    tc::Ring r;
    bool ok = true;
    for (int64_t u = first; u < n_units && ok; u += step) {
      const Unit w = unit_of(g, u);
      const int r0 = (int)(w.rt * L::kRows + rank * 128), c0 = (int)(w.ct * kBN + rank * L::kColsHere);
      for (int k = (int)w.k0; k < (int)w.k1; ++k, ++it, r.next(S)) {
        const uint32_t s = r.s;
        if (!tc::wait(&empty[s], r.phase ^ 1u, fail)) { ok = false; break; }
        if (tc::elect_one()) {
          const uint32_t lb = CTAS == 1 ? 0u : tc::address_in(&full[s], 0);
          // the leader's barrier counts the bytes of both CTAs
          if (rank == 0) mbar_arrive_expect_tx(&full[s], CTAS * (g.a_bytes + L::kB));
          uint8_t *a = sA + s * g.a_bytes, *b = sB + (size_t)s * L::kB;
          const int x = k * kBK;
          if constexpr (A_MN) {
#pragma unroll
            for (int i = 0; i < 2; ++i) load_box<CTAS>(a + i * kBox, &amap, r0 + 64 * i, x, &full[s], lb);
          } else {
            load_box<CTAS>(a, &amap, x, r0, &full[s], lb);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int i = 0; i < L::kColsHere / 64; ++i)
              load_box<CTAS>(b + i * kBox, &bmap, c0 + 64 * i, x, &full[s], lb);
          } else {
#pragma unroll
            for (int i = 0; i < L::kColsHere / 128; ++i)
              load_box<CTAS>(b + i * 2 * kBox, &bmap, x, c0 + 128 * i, &full[s], lb);
          }
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
      // bf16 x bf16 -> fp32; bits 15, 16: operand rows contiguous
      constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((A_MN ? 1u : 0u) << 15) |
                                  ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(kBN >> 3) << 17) |
                                  ((uint32_t)(L::kRows >> 4) << 24);
      const uint32_t a = operand_lo<A_MN>(sA), b = operand_lo<B_MN>(sB);
      uint32_t seg = 0;
      tc::Ring r;
      bool ok = true;
      for (int64_t u = first; u < n_units && ok; u += step) {
        const Unit w = unit_of(g, u);
        if (w.k0 >= w.k1) continue;
        const uint32_t buf = seg & 1u;
        if (!tc::wait(&acc_empty[buf], ((seg >> 1) & 1u) ^ 1u, fail)) break;
        tc::fence_after();
        const uint32_t d = tmem + buf * kBN;
        for (int k = (int)w.k0; k < (int)w.k1; ++k, r.next(S)) {
          const uint32_t s = r.s;
          if (!tc::wait(&full[s], r.phase, fail)) { ok = false; break; }
          tc::fence_after();
          if (tc::elect_one()) {
            const uint32_t sa = a + s * ((uint32_t)g.a_bytes >> 4), sb = b + s * (L::kB >> 4);
#pragma unroll
            for (int i = 0; i < kBK / 16; ++i)
              mma_bf16<CTAS>(d, tc::desc(sa + i * (A_MN ? 2048 >> 4 : 2), tc::kDescSw128Hi),
                             tc::desc(sb + i * (B_MN ? 2048 >> 4 : 2), tc::kDescSw128Hi), kIdesc,
                             (k != (int)w.k0 || i != 0) ? 1u : 0u);
            commit<CTAS>(&empty[s]);
            if (k == (int)w.k1 - 1) commit<CTAS>(&acc_full[buf]);
          }
          __syncwarp();
        }
        ++seg;
      }
      if (*fail) {
        if (tc::elect_one()) commit<CTAS>(&drained);
        mbar_wait(&drained, 0u, tc::kWaitTries);
        bad |= QAMW_STATUS_TIMEOUT;
      }
    }
  } else {
    // a warp takes 32 rows x 128 columns, 32 columns at a time with the next 32 on their way
    const int wq = warp & 3, half = (warp - 2) >> 2;
    const float scale = EPI == kStore ? *g.factor : 1.0f;
    uint32_t seg = 0;
    for (int64_t u = first; u < n_units; u += step) {
      const Unit w = unit_of(g, u);
      const int64_t row = w.rt * L::kRows + rank * 128 + 32 * wq + lane;
      const int64_t col0 = w.ct * kBN + kHalf * half;
      const int n_cols = (int)(g.cols - col0 < kHalf ? g.cols - col0 : kHalf);   // may be <= 0
      const bool in = row < g.rows;
      if (w.k0 >= w.k1) {                  // a split without work: its slot is still a term of the sum
        if constexpr (EPI == kSlot) {
          if (!g.add && in)
            for (int c = 0; c < n_cols; ++c) g.slots[((int64_t)w.split * g.rows + row) * g.cols + col0 + c] = 0.0f;
        }
        continue;
      }
      int tcol = -1;                       // the target's column among this warp's
      float m = -INFINITY;                 // kStats
      float2 sum = make_float2(0.0f, 0.0f);   // of even and odd columns
      float lse = 0.0f, gr = 0.0f;         // kGrad
      if constexpr (EPI == kStats || kIsGrad) {
        const int64_t t = in ? g.targets[row] : g.ignore;
        const bool live = t != g.ignore && t >= 0 && t < g.V;
        const int64_t off = t - (g.v0 + col0);
        if (live && off >= 0 && off < n_cols) tcol = (int)off;
        if constexpr (kIsGrad) {
          lse = in ? g.lse[row] : 0.0f;
          gr = live ? __fdiv_rn(g.grad[row], *g.factor) : 0.0f;
        }
      }
      const uint32_t buf = seg & 1u;
      if (!tc::wait_warp(&acc_full[buf], (seg >> 1) & 1u, fail)) { bad |= QAMW_STATUS_TIMEOUT; break; }
      tc::fence_after();
      uint8_t *tile = sB + S * L::kB + (warp - 2) * tc::kOutBytes;   // this warp's, where the outputs are bf16
      const uint32_t taddr = tmem + buf * kBN + kHalf * half + ((uint32_t)(32 * wq) << 16);
      float buffer[2][32];
      if (n_cols > 0) tc::ld32_async(taddr, buffer[0]);
#pragma unroll
      for (int q = 0; q < kHalf / 32; ++q) {
        const int c = 32 * q;
        if (c >= n_cols) break;
        float(&v)[32] = buffer[q & 1];
        tc::ld_wait();
        tc::tie32(v);
        if (c + 32 < n_cols) tc::ld32_async(taddr + (uint32_t)c + 32, buffer[(q + 1) & 1]);
        const int n = n_cols - c < 32 ? n_cols - c : 32;
        if constexpr (EPI == kStats) {
          if (tcol >= c && tcol < c + 32) {
            float z = 0.0f;   // moved under a predicate: a choice in C++ is made through local memory
#pragma unroll
            for (int j = 0; j < 32; ++j)
              asm volatile("{ .reg .pred p; setp.eq.s32 p, %2, %3; @p mov.f32 %0, %1; }" : "+f"(z) : "f"(v[j]), "r"(tcol - c), "r"(j));
            g.target_logit[row] = z;
          }
          if (n < 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = j < n ? v[j] : -INFINITY;
          }
          float top = v[0];
#pragma unroll
          for (int j = 1; j < 32; ++j) top = fmaxf(top, v[j]);
          // The difference of the logits comes first, then log2 e: neither rounds nor overflows with the logits'
          // own size. A row of -Inf so far has no reference.
          const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.0f : mn;
          const float less = exp2f((m - ref) * kLog2e);
          sum = mul2(sum, make_float2(less, less));
          m = mn;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 d = log2_ratio(v[j], v[j + 1], ref);
            sum = add2(sum, make_float2(exp2f(d.x), exp2f(d.y)));
          }
        } else if constexpr (kIsGrad) {
          const bool none = gr == 0.0f;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 d = log2_ratio(v[j], v[j + 1], lse);
            float p[2] = {exp2f(d.x), exp2f(d.y)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (j + i == tcol - c) p[i] -= 1.0f;
              v[j + i] = none ? 0.0f : gr * p[i];
            }
          }
        }
        if constexpr (EPI == kStore) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= scale;
        }
        if constexpr (EPI == kGradTwo) {
          if (in) {
            __nv_bfloat16 *o = g.out + row * g.ldo + col0 + c;
            tc::store_row32(o, n, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float rest = v[j] - __bfloat162float(__float2bfloat16_rn(v[j]));
              v[j] = fabsf(rest) < INFINITY ? rest : 0.0f;
            }
            tc::store_row32(o + g.rows * g.ldo, n, v);
          }
        } else if constexpr (EPI == kGrad || EPI == kStore) {
          if (g.tma_out) {
            if ((q & 1) == 0) {
              if (lane == 0) tc::stores_read();
              __syncwarp();
            }
            tc::stage_row32(tile, q & 1, v);
            // 64 columns, or the last of them; a warp past the last row has nothing to store
            if (((q & 1) != 0 || c + 32 >= n_cols) && row - lane < g.rows)
              tc::store_tile(tile, &omap, (int)col0 + 32 * (q & ~1), (int)(row - lane));
          } else if (in) {
            tc::store_row32(g.out + row * g.ldo + col0 + c, n, v);
          }
        }
        if constexpr (EPI == kSlot) {
          if (in) {   // cols % 8 == 0: 16-byte groups are all in or all out
            float4 *o = reinterpret_cast<float4 *>(g.slots + ((int64_t)w.split * g.rows + row) * g.cols + col0 + c);
            if (g.add) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (4 * i < n) {
                  const float4 p = o[i];
                  v[4 * i] += p.x, v[4 * i + 1] += p.y, v[4 * i + 2] += p.z, v[4 * i + 3] += p.w;
                }
              }
            }
            tc::store_row32(reinterpret_cast<float *>(o), n, v);
          }
        }
      }
      if constexpr (EPI == kStats)
        if (in && n_cols > 0) g.partials[((g.v0 + col0) / kHalf) * g.rows + row] = make_float2(m, sum.x + sum.y);
      tc::fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CTAS == 1) tc::mbar_arrive(&acc_empty[buf]);
        else tc::arrive_cluster(tc::address_in(&acc_empty[buf], 0));
      }
      ++seg;
    }
    if ((EPI == kGrad || EPI == kStore) && lane == 0) tc::stores_done();
  }

  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if constexpr (CTAS == 2) tc::cluster_sync();   // no CTA leaves while the pair's MMAs, copies or arrivals may reach it
  if (warp == 1) {
    tc::fence_after();
    if constexpr (CTAS == 1) tc::dealloc(tmem, 512);
    else tc::dealloc_pair(tmem, 512);
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) status_or(g.status, bad);
}

// loss and normaliser from the tiles' partial maxima and sums: 32 threads per
// token take every 32nd tile, then join pairwise: a fixed order.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) ce_finish_kernel(const float2 *partials, const float *target_logit,
                                                                   const int64_t *targets, int64_t T, int64_t V,
                                                                   int64_t n_tiles, int64_t ignore, float *loss,
                                                                   float *lse, int32_t *status) {
  __shared__ float2 part[32][33];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * 32 + lane;
  auto join = [](float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * exp2f((a.x - ref) * kLog2e) + b.y * exp2f((b.x - ref) * kLog2e));
  };
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  float2 p = make_float2(-INFINITY, 0.0f);
  if (t < T) {
    for (int64_t i = sl; i < n_tiles; i += 128) {        // four loads in flight
      float2 q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        q[k] = i + 32 * k < n_tiles ? partials[(i + 32 * k) * T + t] : make_float2(-INFINITY, 0.0f);
      const float m = fmaxf(fmaxf(p.x, fmaxf(q[0].x, q[1].x)), fmaxf(q[2].x, q[3].x)), ref = m == -INFINITY ? 0.0f : m;
      float sum = p.y * exp2f((p.x - ref) * kLog2e);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum += q[k].y * exp2f((q[k].x - ref) * kLog2e);
      p = make_float2(m, sum);
    }
  }
  part[sl][lane] = p;
  __syncthreads();
  // warp w joins the 32 terms of token w: lane i holds term i
  p = part[lane][sl];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
    p = join(p, make_float2(__shfl_xor_sync(0xffffffffu, p.x, o), __shfl_xor_sync(0xffffffffu, p.y, o)));
  const int64_t tt = (int64_t)blockIdx.x * 32 + sl;
  if (lane != 0 || tt >= T) return;
  const float n = logf(p.y);
  const int64_t at = targets[tt];
  const bool real = at >= 0 && at < V;
  if (at != ignore && !real) status_or(status, QAMW_STATUS_BAD_INDEX);
  lse[tt] = p.x + n;
  // not lse - target: of a token that the model is sure of, the whole loss lies below a step of lse
  loss[tt] = (at != ignore && real) ? (p.x - target_logit[tt]) + n : 0.0f;
}

// Before the backward pass. CTA 0: the factor of G, max |g| over the tokens that
// count (1 if that is 0, Inf or NaN), and the report of targets out of range. The others: X with the rows of ignored
// tokens set to zero, [T][K], eight columns a thread: their G is zero, but dW =
// G^T X would still turn an Inf or NaN of a padded row into NaN.
__global__ void __launch_bounds__(256) ce_prepare_kernel(const uint4 *X, int64_t ldx8, const int64_t *targets,
                                                         const float *grad, int64_t T, int64_t K8, int64_t V,
                                                         int64_t ignore, int64_t rows, int64_t lo, uint4 *live,
                                                         float *factor, int32_t *status) {
  tc::griddep_launch_dependents();
  auto counts = [&](int64_t t) {
    const int64_t at = targets[t];
    return at != ignore && at >= 0 && at < V;
  };
  if (blockIdx.x == 0) {
    __shared__ uint32_t part[8];
    uint32_t top = 0;   // magnitudes as integers: ordered alike, NaN the largest
    bool bad = false;
    for (int64_t t = threadIdx.x; t < T; t += 256) {
      if (counts(t)) top = max(top, __float_as_uint(grad[t]) & 0x7FFFFFFFu);
      else bad |= targets[t] != ignore;
    }
    if (bad) status_or(status, QAMW_STATUS_BAD_INDEX);
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) top = max(top, part[i]);
      *factor = top == 0u || top >= 0x7F800000u ? 1.0f : __uint_as_float(top);
    }
    return;
  }
  for (int64_t i = (int64_t)(blockIdx.x - 1) * 256 + threadIdx.x; i < rows * K8; i += (int64_t)(gridDim.x - 1) * 256) {
    const int64_t r = i / K8, t = lo > 0 && r >= lo ? r - lo : r;
    live[i] = t < T && counts(t) ? X[t * ldx8 + (i - r * K8)] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// dX = the sum of its terms (`rows` rows apart) times the factor of G, rounded
// to bf16, four columns a thread. GROUPS threads share the terms of a column,
// each every GROUPS-th in order, and the first adds theirs in order: few tokens
// have many terms and few columns (16 x 2048, 36 terms: 11.6 us with one thread
// a column).
template <int GROUPS>
__global__ void __launch_bounds__(256) ce_sum_slots_kernel(const float *slots, int terms, int64_t rows,
                                                           const float *factor, int64_t T, int64_t K,
                                                           __nv_bfloat16 *dX, int64_t ldx) {
  constexpr int kCols = 256 / GROUPS;
  __shared__ float4 part[GROUPS][kCols];
  const int c = threadIdx.x % kCols, group = threadIdx.x / kCols;
  const int64_t n = T * K / 4;
  const float f = *factor;
  for (int64_t i0 = (int64_t)blockIdx.x * kCols; i0 < n; i0 += (int64_t)gridDim.x * kCols) {
    const int64_t i = i0 + c;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4 &b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; };
    if (i < n) {
#pragma unroll 8
      for (int s = group; s < terms; s += GROUPS) add(reinterpret_cast<const float4 *>(slots + s * rows * K)[i]);
    }
    if constexpr (GROUPS > 1) {
      part[group][c] = a;
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int g = 1; g < GROUPS; ++g) add(part[g][c]);
      }
      __syncthreads();
    }
    if (group != 0 || i >= n) continue;
    const int64_t row = 4 * i / K, col = 4 * i - row * K;
    __nv_bfloat16 *o = dX + row * ldx + col;
    const __nv_bfloat162 p = __floats2bfloat162_rn(a.x * f, a.y * f), q = __floats2bfloat162_rn(a.z * f, a.w * f);
    if (reinterpret_cast<uintptr_t>(o) % 8 == 0) {
      *reinterpret_cast<uint2 *>(o) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&p), *reinterpret_cast<const uint32_t *>(&q));
    } else {
      o[0] = p.x, o[1] = p.y, o[2] = q.x, o[3] = q.y;
    }
  }
}

// [rows][cols] bf16 in memory, boxes of box_c x box_r
bool make_map(CUtensorMap *m, const void *p, int64_t rows, int64_t cols, int64_t ld, int box_r, int box_c) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {(cuuint32_t)box_c, (cuuint32_t)box_r};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
  const void *p;
  int64_t rows, cols, ld;         // as it lies in memory
};

template <int CTAS, bool A_MN, bool B_MN, int EPI>
cudaError_t run(const Operand &A, const Operand &B, CeArgs g, cudaStream_t s) {
  using L = CeTile<CTAS>;
  // At most 120 rows: only they (in eights) are loaded, which leaves room for
  // more stages; the MMA reads what follows them in shared memory as rows whose
  // results no one looks at. (16 tokens x 32000 x 2048: filling the other 112
  // rows with zeros took 5 of 38 us.)
  const int a_rows = A_MN || CTAS == 2 ? 128 : (int)std::min<int64_t>(128, (g.rows + 7) / 8 * 8);
  g.a_bytes = a_rows * 128;
  CUtensorMap amap, bmap;
  if (!make_map(&amap, A.p, A.rows, A.cols, A.ld, A_MN ? 64 : a_rows, 64) ||
      !make_map(&bmap, B.p, B.rows, B.cols, B.ld, B_MN ? 64 : 128, 64))
    return cudaErrorInvalidValue;
  int dev = 0, smem_max = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&smem_max, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess) return e;
  g.n_r = (g.rows + L::kRows - 1) / L::kRows;
  g.n_c = (g.cols + kBN - 1) / kBN;
  // A lane holds a row of the accumulator, and 32 lanes that store to 32 rows
  // keep the L1 pipe busy (69% in dW of 301 tokens). Where a tile has few steps,
  // bf16 outputs are laid out in shared memory and leave by TMA stores instead
  // (gradient of 16 tokens x 32000 x 2048 99 -> 91 us, of 128 tokens 109 -> 101);
  // with more steps the stage of loads that this memory costs is worth more (512
  // tokens 177 -> 183, 4096 x 65536 x 4096 4.11 -> 4.17 ms).
  CUtensorMap omap = amap;
  const bool bf16_out = (EPI == kGrad || EPI == kStore) && g.depth <= kShortDepth;
  g.tma_out = bf16_out && reinterpret_cast<uintptr_t>(g.out) % 16 == 0 && g.ldo % 8 == 0;
  if (g.tma_out && !make_map(&omap, g.out, g.rows, g.cols, g.ldo, 32, 64)) return cudaErrorInvalidValue;
  const int64_t out_bytes = bf16_out ? 8 * tc::kOutBytes : 0;
  g.stages = (int)std::min<int64_t>(kMaxStages, (smem_max - 2048 - out_bytes) / (g.a_bytes + L::kB));
  const size_t smem = 1024 + (size_t)g.stages * (g.a_bytes + L::kB) + (size_t)out_bytes;
  auto kern = ce_gemm_kernel<CTAS, A_MN, B_MN, EPI>;
  if ((e = set_max_dynamic_smem(reinterpret_cast<const void *>(kern), smem)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(CTAS * std::min<int64_t>(sm_count() / CTAS, g.n_r * g.n_c * g.splits)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CTAS;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set up beside the kernel before this one
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, amap, bmap, omap, g);
}

// One CTA per tile, or a pair. A step of either takes the same time, so the
// fewer waves win; the pair does on a tie, since it loads a third less (4096
// tokens x 32000 x 4096: 670 us in pairs, 830 in single CTAs; gradient of 301
// tokens x 50021 x 2048: 256 in pairs, 236 by this rule). A contraction of at
// most 8 steps is bound by its epilogue, which single CTAs overlap better (the
// same gradient with dW in single CTAs: 225; of 768 tokens, 12 steps: 235 in
// pairs, 243).
bool single_cta(int64_t rows, int64_t depth, int64_t tiles_c) {
  if (depth <= 8 * kBK) return true;
  const int64_t one = ((rows + 127) / 128) * tiles_c, pair = ((rows + 255) / 256) * tiles_c;
  const int64_t sms = sm_count();
  return (one + sms - 1) / sms < (pair + sms / 2 - 1) / (sms / 2);
}
template <bool A_MN, bool B_MN, int EPI>
cudaError_t run_rows(const Operand &A, const Operand &B, const CeArgs &g, cudaStream_t s) {
  const int64_t tiles_c = (g.cols + kBN - 1) / kBN * g.splits;
  return single_cta(g.rows, g.depth, tiles_c) ? run<1, A_MN, B_MN, EPI>(A, B, g, s)
                                              : run<2, A_MN, B_MN, EPI>(A, B, g, s);
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int64_t vocab_tiles(int64_t V) { return (V + kHalf - 1) / kHalf; }   // that have a partial maximum and sum

// Contraction splits of dX for pieces of `piece` vocabulary entries: the number
// up to 32, each split at least 8 steps long, with the least waves x (steps + 4).
int dx_splits(int64_t T, int64_t K, int64_t piece) {
  const int64_t tiles_c = (K + kBN - 1) / kBN, steps = (piece + kBK - 1) / kBK, sms = sm_count();
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 32 && (s == 1 || steps / s >= 8); ++s) {
    const int ctas = single_cta(T, piece, tiles_c * s) ? 1 : 2;
    const int64_t units = ((T + 128 * ctas - 1) / (128 * ctas)) * tiles_c * s;
    const int64_t cost = (units + sms / ctas - 1) / (sms / ctas) * ((steps + s - 1) / s + 4);
    if (cost < least) best = s, least = cost;
  }
  return best;
}

}  // namespace

CeWorkspace ce_workspace(int64_t T, int64_t V) {
  CeWorkspace w;
  w.target_logit = align256((size_t)vocab_tiles(V) * (size_t)T * sizeof(float2));
  w.total = w.target_logit + align256((size_t)T * 4);
  return w;
}

// Up to 16 tokens G is held as two bf16 terms, rows t and lo + t of a matrix of
// 2 lo rows: the tiles have room for both, so the products cost no more MMAs.
// With so few tokens the rounding of one term would show: gradients were off by
// up to 0.57% (one token) and by 1.9 times what their bf16 outputs cannot avoid.
// From 17 tokens on it averages out (1.25 times at most in 12 thousand random
// cases). 32000 x 2048, dX and dW / dX alone: 1 token 96 / 52 us (one term 95 /
// 50), 16 tokens 94 / 55 (96 / 51); at 64 tokens two terms took 107 / 68 us, one
// 94 / 56.
constexpr int64_t kTwoTerms = 16;

CeGradWorkspace ce_grad_workspace(int64_t T, int64_t K, int64_t piece) {
  CeGradWorkspace w;
  w.ldg = (piece + 7) / 8 * 8;
  w.lo = T <= kTwoTerms ? T : 0;
  w.rows = T + w.lo;
  w.live = align256((size_t)w.rows * (size_t)w.ldg * 2);
  w.factor = w.live + align256((size_t)w.rows * (size_t)K * 2);
  w.slots = w.factor + 256;
  w.splits = dx_splits(w.rows, K, piece);
  w.total = w.slots + align256((size_t)w.splits * (size_t)w.rows * (size_t)K * 4);
  return w;
}

cudaError_t launch_ce_piece(const CeArgsIn &a, void *workspace, cudaStream_t s) {
  const CeWorkspace w = ce_workspace(a.T, a.V);
  CeArgs g = {};
  g.rows = a.T;
  g.cols = a.n;
  g.depth = a.K;
  g.splits = 1;
  g.steps_per_split = (a.K + kBK - 1) / kBK;
  g.status = a.status;
  g.targets = a.targets;
  g.v0 = a.v0;
  g.V = a.V;
  g.ignore = a.ignore;
  g.partials = static_cast<float2 *>(workspace);
  g.target_logit = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + w.target_logit);
  return run_rows<false, false, kStats>({a.X, a.T, a.K, a.ldx}, {a.W, a.n, a.K, a.ldw}, g, s);
}

cudaError_t launch_ce_finish(const CeArgsIn &a, void *workspace, float *loss, float *lse, cudaStream_t s) {
  const CeWorkspace w = ce_workspace(a.T, a.V);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + 31) / 32), 1, 1);
  cfg.blockDim = dim3(kFinishThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ce_finish_kernel, static_cast<const float2 *>(workspace),
                            reinterpret_cast<const float *>(static_cast<unsigned char *>(workspace) + w.target_logit),
                            a.targets, a.T, a.V, vocab_tiles(a.V), a.ignore, loss, lse, a.status);
}

cudaError_t launch_ce_grad_piece(const CeArgsIn &a, const float *lse, const float *grad, int64_t piece, bool first,
                                 void *dW, int64_t lddw, void *workspace, cudaStream_t s) {
  const CeGradWorkspace w = ce_grad_workspace(a.T, a.K, piece);
  __nv_bfloat16 *G = static_cast<__nv_bfloat16 *>(workspace);
  uint4 *live = reinterpret_cast<uint4 *>(static_cast<unsigned char *>(workspace) + w.live);
  float *factor = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + w.factor);
  if (first) {
    const int64_t blocks = (w.rows * a.K / 8 + 255) / 256, most = (int64_t)sm_count() * 16;
    ce_prepare_kernel<<<(unsigned)(1 + std::min(blocks, most)), 256, 0, s>>>(
        static_cast<const uint4 *>(a.X), a.ldx / 8, a.targets, grad, a.T, a.K / 8, a.V, a.ignore, w.rows,
        w.lo, live, factor, a.status);
    const cudaError_t c = cudaGetLastError();
    if (c != cudaSuccess) return c;
  }
  const Operand X{live, w.rows, a.K, a.K}, Gm{G, w.rows, a.n, w.ldg};
  CeArgs g = {};
  g.rows = a.T;
  g.cols = a.n;
  g.depth = a.K;
  g.splits = 1;
  g.steps_per_split = (a.K + kBK - 1) / kBK;
  g.status = a.status;
  g.targets = a.targets;
  g.v0 = a.v0;
  g.V = a.V;
  g.ignore = a.ignore;
  g.lse = lse;
  g.grad = grad;
  g.factor = factor;
  g.out = G;
  g.ldo = w.ldg;
  const Operand W{a.W, a.n, a.K, a.ldw};
  cudaError_t e = w.lo > 0 ? run_rows<false, false, kGradTwo>(X, W, g, s) : run_rows<false, false, kGrad>(X, W, g, s);
  if (e != cudaSuccess) return e;
  CeArgs x = {};
  x.rows = w.rows;
  x.cols = a.K;
  x.depth = a.n;
  x.splits = w.splits;
  x.steps_per_split = ((a.n + kBK - 1) / kBK + w.splits - 1) / w.splits;
  x.status = a.status;
  x.slots = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + w.slots);
  x.add = first ? 0 : 1;
  if ((e = run_rows<false, true, kSlot>(Gm, W, x, s)) != cudaSuccess) return e;
  if (dW == nullptr) return cudaSuccess;
  CeArgs d = {};
  d.rows = a.n;
  d.cols = a.K;
  d.depth = w.rows;
  d.splits = 1;
  d.steps_per_split = (w.rows + kBK - 1) / kBK;
  d.status = a.status;
  d.factor = factor;
  d.out = static_cast<__nv_bfloat16 *>(dW);
  d.ldo = lddw;
  return run_rows<true, true, kStore>(Gm, X, d, s);
}

cudaError_t launch_ce_grad_finish(int64_t T, int64_t K, int64_t piece, void *dX, int64_t lddx, void *workspace,
                                  cudaStream_t s) {
  const CeGradWorkspace w = ce_grad_workspace(T, K, piece);
  const int terms = w.lo > 0 ? 2 * w.splits : w.splits;
  // one thread a column while that gives every SM a block (64 x 4096, 9 terms: 189 us of gradient, 193 shared)
  const int groups = terms >= 8 && T * K / 4 < 256 * (int64_t)sm_count() ? 8 : 1;
  const int64_t blocks = (T * K / 4 * groups + 255) / 256, most = (int64_t)sm_count() * 16;
  auto run = [&](auto kernel) {
    kernel<<<(unsigned)std::min(blocks, most), 256, 0, s>>>(
        reinterpret_cast<const float *>(static_cast<unsigned char *>(workspace) + w.slots), terms, w.lo > 0 ? w.lo : T,
        reinterpret_cast<const float *>(static_cast<unsigned char *>(workspace) + w.factor), T, K,
        static_cast<__nv_bfloat16 *>(dX), lddx);
  };
  if (groups == 8) run(ce_sum_slots_kernel<8>);
  else run(ce_sum_slots_kernel<1>);
  return cudaGetLastError();
}

}  // namespace qamw
