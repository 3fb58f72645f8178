// qamw_tcgen05.cuh -- the pieces that the tensor-core kernels of
// qamw_mx4_gemm.cu and qamw_cross_entropy.cu share: shared-memory operand
// descriptors, TMA tile loads, MMA issue and commit, tensor-memory loads, and
// waits that are bounded and give up together.
#pragma once

#include <cstdint>

#include "qamw_device.cuh"
#include "qamw_mbarrier.cuh"
#include "qamw_tensor_map.h"

namespace qamw {
namespace tc {

constexpr uint32_t kWaitTries = 1u << 22;   // try_wait attempts before a wait gives up

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

// Loads and MMAs are issued by one lane of a warp whose 32 lanes walk the loop
// together: the operands of these instructions are uniform registers, and only
// in code that the compiler sees to be uniform are they formed without a
// detour for every instruction (with the loop inside `if (lane == 0)` a stage
// of the 4-bit kernels took 1.0 us, its MMAs 0.27).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
  return p != 0u;
}

// Bounded wait of a whole warp, one answer for all lanes: true once the phase
// has completed. It gives up, and raises the CTA's failure flag, after
// kWaitTries attempts, and gives up early once another role has raised it:
// every role then leaves its loop.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *fail) {
  for (uint32_t i = 0; i < kWaitTries; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63u) == 63u && __any_sync(0xffffffffu, *fail != 0)) return false;
  }
  *fail = 1;
  return false;
}

// The same for a whole warp that waits long (an epilogue for its accumulators):
// one lane asks, and sleeps between its attempts, so that the waiting takes
// nothing from the warps that load and multiply.
constexpr uint32_t kSleepTries = 1u << 22;   // attempts, at most 128 ns apart
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *fail) {
  int ok = 0;
  if ((threadIdx.x & 31) == 0) {
    uint32_t ns = 32;
    for (uint32_t i = 0; i < kSleepTries; ++i) {
      if (mbar_try_wait(bar, parity)) { ok = 1; break; }
      if (*fail) break;
      __nanosleep(ns);
      if (ns < 128) ns <<= 1;
    }
    if (!ok) *fail = 1;
  }
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The place in a ring of `n` stages: index and phase, stepped without a
// division (one costs a stage of the 4-bit kernels a tenth of its time).
struct Ring {
  uint32_t s = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t n) {
    if (++s == n) s = 0, phase ^= 1u;
  }
};

// Operand descriptors: the low word holds the address / 16, so that stages and
// steps inside a stage are additions to it.
// 128-byte swizzle, K contiguous: rows of 128 bytes, 8-row atoms 1024 bytes
// apart (the leading offset is unused in this layout).
constexpr uint32_t kDescSw128Hi = (uint32_t)(1024 >> 4) | (1u << 14) | (2u << 29);
// No swizzle, 16-byte rows, 8-row atoms of 128 contiguous bytes (scale tiles
// for tcgen05.cp).
constexpr uint32_t kDescScalesHi = (uint32_t)(128 >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_lo(const void *p, uint32_t leading = 1) {
  return (smem_u32(p) >> 4) | (leading << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// One TMA tile (x: innermost coordinate in elements, y: row) into shared memory.
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// `bytes` contiguous bytes (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void load_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// ---- clusters and CTA pairs (cta_group::2) ----
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the address of this CTA's shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t address_in(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// A tile into this CTA's memory, counted at the barrier `bar` (a cluster
// address) of either CTA of the pair.
__device__ __forceinline__ void load_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// to the barrier at this place in both CTAs of the pair
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t *slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

// ---- programmatic dependent launch ----
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void griddep_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;"); }

// The walk over n_r x n_c tiles: groups of `group` row tiles, the row varying
// fastest inside a group, so that the row operand of a group stays in L2 while
// the columns go by.
struct TileWalk {
  int64_t n_r, n_c, group;
  __device__ __forceinline__ void at(int64_t t, int64_t &rt, int64_t &ct) const {
    const int64_t per = group * n_c, g = t / per, in = t - g * per;
    const int64_t left = n_r - g * group, h = left < group ? left : group;
    ct = in / h;
    rt = g * group + (in - ct * h);
  }
};

// 32 contiguous outputs of a lane's row, `n` of them real: whole 32-byte sectors
// where the address allows it (two 16-byte stores per sector double the
// requests to L2), single values at a ragged end.
__device__ __forceinline__ void store_32b(void *p, const uint32_t *w) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
               : "memory");
}
__device__ __forceinline__ void store_row32(float *o, int n, const float *v) {
  if (n >= 32 && reinterpret_cast<uintptr_t>(o) % 32 == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
      store_32b(o + 8 * i, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) o[j] = v[j];
  }
}
__device__ __forceinline__ void store_row32(__nv_bfloat16 *o, int n, const float *v) {
  if (n >= 32 && reinterpret_cast<uintptr_t>(o) % 16 == 0) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if (reinterpret_cast<uintptr_t>(o) % 32 == 0) {
      store_32b(o, w);
      store_32b(o + 16, w + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint4 *>(o)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) o[j] = __float2bfloat16_rn(v[j]);
  }
}

// ---- tiles back to device memory (a warp's 32 rows x 64 bf16 columns) ----
constexpr int kOutBytes = 32 * 128;   // 128-byte swizzle: 16-byte piece p of row r lies at piece p ^ (r % 8)
// 32 columns of the lane's row: pieces 4 * half .. 4 * half + 3
__device__ __forceinline__ void stage_row32(uint8_t *tile, int half, const float *v) {
  const int r = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(tile + r * 128 + (((4 * half + i) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The warp's tile out by one TMA store (rows and columns past the tensor's end
// are not written); by all lanes, once they have written the tile.
__device__ __forceinline__ void store_tile(const uint8_t *tile, const CUtensorMap *map, int x, int y) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
                 "r"(y), "r"(smem_u32(tile))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
// until the lane's stores have read their tiles / are done
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Tensor-memory allocation by one whole warp; `cols` a power of two >= 32.
__device__ __forceinline__ void alloc(uint32_t *slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t tmem, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols) : "memory");
}

__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// 32 consecutive accumulator columns of the warp's 32 lanes, valid after ld_wait()
__device__ __forceinline__ void ld32_async(uint32_t taddr, float *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr)
      : "memory");
}
// After ld_wait(): the values of an ld32_async are used from here on (the
// compiler sees no other reason to keep their uses below the wait).
__device__ __forceinline__ void tie32(float *v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
// 16 consecutive accumulator columns of the warp's 32 lanes
__device__ __forceinline__ void ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
  ld_wait();
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]),
                 "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}

}  // namespace tc
}  // namespace qamw
