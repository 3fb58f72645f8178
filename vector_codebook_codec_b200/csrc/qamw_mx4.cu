// qamw_mx4.cu -- microscaled 4-bit floating point (OCP MX: e2m1 elements, one
// power-of-two scale per 32 columns): quantisation and decode, after the
// codec's own preparation of a row (Methodology (5) Activation-Aware Scaling
// and (2) Deterministic Rotation).
//
//   v_j = w_j s_j  or  w_j / s_j;   y = H_b (d (.) v) / sqrt(b)  per block of b columns
//   e   = clamp(floor(log2 max|y|) - 2, -127, 127) per group of 32 columns
//   q_j = the e2m1 value nearest y_j 2^-e (ties to the even code, at most 6)
//
// The result is that of fp64 arithmetic with no rounding before the 4-bit
// decision, but the work is done in fp32: a value is computed with a bound m on
// its error, and both y - m and y + m are rounded to 4 bits. Where they agree,
// so does every value between them, the exact one among them. Where they
// differ (about 6 in 10^5 values of Gaussian rows at b = 128), or the group's
// exponent hangs on the error, or the group is so small beside its block that
// m is not small beside its values (64 m above its largest), the warp forms the
// values in fp64 from the row.
// An e2m1 border has at most three significant bits, so the exponent and the
// top mantissa bits of that double, with a sticky bit for the rest, decide
// exactly (double_scaled).
//
// Error of the fp32 value, with A = sum of |v| over the block: v itself 2 x
// 2^-24 (1/s rounded, and the product), one rounding of at most 2^-24 A per
// butterfly level, the factor 2^-e / sqrt(b) one and the sum y +- m, fused with
// its product, one more: (log2 b + 4) 2^-24 A. A <= sqrt(b sum v^2) takes its
// place: half the instructions, 1.25 times as large for Gaussian rows. The
// factor used is log2 b + 6: the bound's own roundings are 10^-6 of it.
//
// A lane loads two runs of 16 columns, 64 columns apart, so that four lanes
// read 128 contiguous bytes of bf16; block bits 0-3 and 6 are butterflies on
// its registers (two columns an instruction), bits 4, 5 and 7-9 exchanges
// between lanes. A group of 32 columns is one run of two neighbour lanes.
#include <type_traits>

#include <cuda_fp16.h>

#include "qamw_device.cuh"
#include "qamw_internal.h"

namespace qamw {
namespace {

constexpr int kMxWarps = 4;         // warps per CTA
// Warps that an SM is meant to hold: 16 (128 registers) for the quantisation of
// prepared rows (11008 x 4096 bf16, b = 128, before its rows were taken in turn: 71 us,
// 20 warps the same, 24 spill: 84),
// and for decoding rotated ones, 24 for the kernels that neither bound an error
// nor rotate (values of the same matrix decoded: 29 us at 16, 27 at 24).
constexpr int kMxResident = 16, kMxResidentPlain = 24;
constexpr int kMxUnit = 1024;       // columns per warp pass: 32 lanes x 32 columns

// Byte offset of the scale of (row, group) in the tiled layout: tiles of 128
// rows x 4 groups, 512 bytes each, row tiles outermost; inside a tile row r
// and group g sit at (r % 32) * 16 + (r / 32) * 4 + g, the order in which the
// tensor cores take scale factors.
__device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t group, int64_t k_tiles) {
  const int r = (int)(row & 127);
  return ((row >> 7) * k_tiles + (group >> 2)) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (group & 3);
}

// eight floats -> eight e2m1 codes (round to nearest even, saturating), v[0] in the low bits
__device__ __forceinline__ uint32_t e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// eight e2m1 codes -> four pairs of fp16 (exact)
__device__ __forceinline__ void halves_of_e2m1x8(uint32_t w, uint32_t *h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(b - 127) for a scale byte: 0 is the subnormal 2^-127, 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// y 2^-e as a float for the 4-bit rounding: truncated, with the lowest bit set
// if anything was cut off. Values below 2^-126 become 0 (they round to code 0:
// the lowest border is 2^-2); values beyond the fp32 range (e clamped at 127)
// become the largest float (code 6).
__device__ __forceinline__ float double_scaled(double y, int e) {
  const uint64_t b = (uint64_t)__double_as_longlong(y);
  const uint32_t hi = (uint32_t)(b >> 32), lo = (uint32_t)b;
  const int ex = (int)((hi >> 20) & 0x7FFu) - e - (1023 - 127);   // fp32 exponent field
  uint32_t m = ((hi & 0xFFFFFu) << 3) | (lo >> 29) | ((lo & 0x1FFFFFFFu) ? 1u : 0u);
  m |= (uint32_t)ex << 23;
  if (ex <= 0) m = 0u;
  if (ex >= 255) m = 0x7F7FFFFFu;
  return __uint_as_float(m | (hi & 0x80000000u));
}

struct MxQuantArgs {
  const void *W;
  int64_t M, K, ldw;
  const float *s;       // [K] or nullptr
  int divide;
  int log2b;            // 0: no rotation
  uint64_t seed;
  uint8_t *codes;       // [M][K/2]
  uint8_t *scales;      // tiled
  int32_t *status;
  int64_t units_k;      // column units
  int64_t row_groups;   // rows of a unit are dealt out to row_groups warps
  int vec;              // widest loads allowed: 32, 16 or 0 bytes
};

// 32 contiguous bytes
__device__ __forceinline__ void load_32b(const void *p, int vec, uint32_t (&w)[8]) {
  if (vec == 32) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = static_cast<const uint4 *>(p)[0], b = static_cast<const uint4 *>(p)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store_32b(void *p, int vec, const uint32_t (&w)[8]) {
  if (vec == 32) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
    static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A row's words of the lane: 16 columns from p, bf16 (8 words) or fp32 (16).
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ float value(const uint32_t *w, int j) {
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
  }
  static __device__ __forceinline__ double exact(const void *p, int64_t i) {
    return bf16_bits_to_double(static_cast<const uint16_t *>(p)[i]);
  }
};
template <>
struct Raw<float> {
  static constexpr int kWords = 16;
  static __device__ __forceinline__ float value(const uint32_t *w, int j) { return __uint_as_float(w[j]); }
  static __device__ __forceinline__ double exact(const void *p, int64_t i) {
    return (double)static_cast<const float *>(p)[i];
  }
};
template <typename T>
__device__ __forceinline__ void load16(const T *p, int vec, bool in, uint32_t *w) {
  constexpr int N = Raw<T>::kWords;
  if (!in) {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 0u;
  } else if (vec) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      uint32_t q[8];
      load_32b(reinterpret_cast<const uint8_t *>(p) + 32 * i, vec, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[8 * i + j] = q[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (N == 8) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
      else w[i] = __float_as_uint(p[i]);
    }
  }
}

// What decide_exactly found: code words and the masks of the codes decided.
struct Decided {
  uint32_t code[4], mask[4];
  int e;
  bool finite;
};

// A group's 32 values in fp64, lane k forming y of its column k: the block's
// v_i are loaded once, 32 at a time, and handed round,
//   y_k = sum_i (-1)^popc(i & k) d_i v_i / sqrt(b).
// Then the codes of the values of `mask` at the exponent e; with all of them
// (mask ~0) the group's exponent is found too. Warp-collective.
template <typename T>
__device__ __noinline__ Decided decide_exactly(const MxQuantArgs &p, int64_t row, int64_t group, uint32_t mask, int e) {
  const int lane = threadIdx.x & 31, b = 1 << p.log2b;
  const int64_t base = (32 * group) & ~(int64_t)((b > 32 ? b : 32) - 1);
  const int local = (int)(32 * group - base);            // of the group in its block (0 for b <= 32)
  const void *w = static_cast<const T *>(p.W) + row * p.ldw;
  uint32_t flip = 0;                                      // bit i: the sign of v_i in y_lane
  for (int i = 0; i < 32; ++i) flip |= (uint32_t)(__popc(i & lane & (b - 1)) & 1) << i;
  double y0 = 0.0, y1 = 0.0;
  for (int q = 0; q < (b > 32 ? b : 32); q += 32) {
    const int64_t c = base + q + lane;
    double v = Raw<T>::exact(w, c);
    if (p.s != nullptr) v = p.divide ? v / (double)p.s[c] : v * (double)p.s[c];
    if (p.log2b > 0 && mask_is_negative(p.seed, c)) v = -v;
    const uint32_t f = (__popc(q & local) & 1) ? ~flip : flip;
    if (b >= 32) {
#pragma unroll 8
      for (int i = 0; i < 32; i += 2) {
        const double s0 = __shfl_sync(0xffffffffu, v, i), s1 = __shfl_sync(0xffffffffu, v, i + 1);
        y0 += ((f >> i) & 1u) ? -s0 : s0;
        y1 += ((f >> (i + 1)) & 1u) ? -s1 : s1;
      }
    } else {                                              // several blocks in a group: the lane's own
      for (int i = 0; i < 32; ++i) {
        const double s0 = __shfl_sync(0xffffffffu, v, i);
        if ((i >> p.log2b) == (lane >> p.log2b)) y0 += ((f >> i) & 1u) ? -s0 : s0;
      }
    }
  }
  double y = y0 + y1;
  if (p.log2b > 0) y *= 1.0 / sqrt((double)b);
  Decided d;
  d.e = e;
  d.finite = true;
  if (mask == 0xffffffffu) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, (uint32_t)__double2hiint(y) & 0x7FFFFFFFu);
    d.finite = top < 0x7FF00000u;
    d.e = min(max((int)(top >> 20) - 1023 - 2, -127), 127);
  }
  const float one[8] = {d.finite ? double_scaled(y, d.e) : 0.0f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool own = (mask >> lane) & 1u;
  uint32_t n = own ? (e2m1x8(one) & 15u) << (4 * (lane & 7)) : 0u;     // this value's code, in its place
  uint32_t m = own ? 15u << (4 * (lane & 7)) : 0u;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    n |= __shfl_xor_sync(0xffffffffu, n, o);
    m |= __shfl_xor_sync(0xffffffffu, m, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    d.code[i] = __shfl_sync(0xffffffffu, n, 8 * i);
    d.mask[i] = __shfl_sync(0xffffffffu, m, 8 * i);
  }
  return d;
}

// The lane's place in a unit of 1024 columns: column bits 4 and 5 are lane bits
// 0 and 1, bit 6 its two runs, bits 7-9 lane bits 2-4.
struct LanePlace {
  int64_t run0;    // first column of run 0; run 1 starts 64 columns on
  int64_t group0;  // the group of run 0; run 1's is the second next
  __device__ __forceinline__ LanePlace(int64_t unit, int lane) {
    run0 = unit * kMxUnit + 128 * (lane >> 2) + 32 * ((lane >> 1) & 1) + 16 * (lane & 1);
    group0 = run0 / 32;
  }
};

__device__ __forceinline__ float2 diff2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

// the largest magnitude of three (NaNs left out)
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// block bits 0-3: column bits 0-3 are the index j of the array
__device__ __forceinline__ void butterflies_low(float2 (&x)[16], int log2b) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if (t < log2b) {
      const int h = 1 << t;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if ((j & h) == 0) {
          const float2 a = x[j], b = x[j | h];
          x[j] = add2(a, b);
          x[j | h] = diff2(a, b);
        }
      }
    }
  }
}
// the bit that separates the two halves of every pair
__device__ __forceinline__ void butterflies_pair(float2 (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = make_float2(x[j].x + x[j].y, x[j].x - x[j].y);
}
// a bit that is lane bit `h`
__device__ __forceinline__ void butterflies_lane(float2 (&x)[16], int lane, int h) {
  const float s = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, x[j].x, h), __shfl_xor_sync(0xffffffffu, x[j].y, h));
    x[j] = fma2(x[j], make_float2(s, s), o);
  }
}

// Column factors of a unit, formed once by the CTA (its warps work on rows of
// one unit) and kept in shared memory as the lanes read them: 8 x 32 float4,
// (run 0, run 1) of columns 2i and 2i + 1 of a lane.
using Factors = float4[8][32];
__device__ __forceinline__ float2 factor(const Factors &f, int lane, int j) {
  const float4 q = f[j >> 1][lane];
  return (j & 1) ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
}
template <typename F>
__device__ __forceinline__ void form_factors(Factors &f, int64_t unit, int64_t K, F of) {
#pragma unroll
  for (int n = 0; n < kMxUnit / (32 * kMxWarps); ++n) {   // a fixed count: the loads of s go out together
    const int i = threadIdx.x + n * 32 * kMxWarps;
    const int64_t col = unit * kMxUnit + i;
    const int lane = 4 * (i >> 7) + ((i >> 4) & 3), j = i & 15, run = (i >> 6) & 1;
    reinterpret_cast<float *>(&f[j >> 1][lane])[2 * (j & 1) + run] = col < K ? of(col) : 1.0f;
  }
  __syncthreads();
}

// Every butterfly of a block of 2^LB columns on the lane's 2 x 16 columns.
template <int LB>
__device__ __forceinline__ void rotate(float2 (&x)[16], int lane) {
  butterflies_low(x, LB);
  if constexpr (LB > 6) butterflies_pair(x);
  if constexpr (LB > 4) butterflies_lane(x, lane, 1);
  if constexpr (LB > 5) butterflies_lane(x, lane, 2);
#pragma unroll
  for (int t = 7; t < LB; ++t) butterflies_lane(x, lane, 1 << (t - 5));
}

// PREP: a channel scale or a rotation (blocks of 2^LB columns); otherwise the
// values are exact as read. 11008 x 4096 bf16: 60 us at b = 128 with a scale
// (1.9 TB/s; 784 instructions per 1024 values, 245 of them on the integer pipe at
// half rate, 14 warps per SM, 60% of the issue slots; 66 us with the rows dealt
// out beforehand), 23 us plain (5 TB/s).
template <typename T, bool PREP, int LB>
__global__ void __launch_bounds__(32 * kMxWarps, (PREP ? kMxResident : kMxResidentPlain) / kMxWarps)
    mx4_quantize_kernel(const __grid_constant__ MxQuantArgs p) {
  constexpr int N = Raw<T>::kWords;
  const int lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x % p.units_k, first = blockIdx.x / p.units_k, ctas = p.row_groups / kMxWarps;
  // The CTA's rows are first, first + ctas, ...; its warps take them in turn as
  // they come free, since a row that needs fp64 takes several times as long.
  __shared__ int taken;
  if (threadIdx.x == 0) taken = kMxWarps;
  const int64_t rg = first + (threadIdx.x >> 5) * ctas;
  const LanePlace at(unit, lane);
  const int64_t k_tiles = (p.K + 127) / 128, rows_pad = (p.M + 127) / 128 * 128;
  // K % 32 == 0: a run of 16 columns and a group are all in or all out
  const bool in[2] = {at.run0 < p.K, at.run0 + 64 < p.K};
  const T *src = static_cast<const T *>(p.W) + at.run0;
  // the product of mx4_linear may start: it waits for this kernel before it reads the codes
  asm volatile("griddepcontrol.launch_dependents;");
  uint32_t w0[N], w1[N];
  if (rg < p.M) {
    load16<T>(src + rg * p.ldw, p.vec, in[0], w0);
    load16<T>(src + rg * p.ldw + 64, p.vec, in[1], w1);
  }
  __shared__ Factors f;
  if (PREP)   // +-s, +-1/s or +-1; one far from 1 becomes NaN: its rows are decided from fp64
    form_factors(f, unit, p.K, [&](int64_t col) {
      float v = 1.0f;
      if (p.s != nullptr) {
        v = p.divide ? __frcp_rn(p.s[col]) : p.s[col];
        if (!(fabsf(v) > 0x1p-100f && fabsf(v) < 0x1p100f)) v = __uint_as_float(0x7FC00000u);
      }
      return (LB > 0 && mask_is_negative(p.seed, col)) ? -v : v;
    });
  const float inv = (float)(1.0 / sqrt((double)(1 << LB)));
  uint32_t bad = 0;
  if (!PREP) __syncthreads();   // `taken` is set (form_factors ends with a barrier too)
  int64_t next;
  for (int64_t row = rg; row < rows_pad; row = next) {
    int turn = 0;
    if (lane == 0) turn = atomicAdd(&taken, 1);
    next = first + (int64_t)__shfl_sync(0xffffffffu, turn, 0) * ctas;
    uint32_t sword = 0;
    if (row < p.M) {
      float2 x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = make_float2(Raw<T>::value(w0, j), Raw<T>::value(w1, j));
      uint32_t any0 = 0, any1 = 0;    // nonzero bits of each run, signs apart
      if (PREP) {
        const uint32_t drop = N == 8 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
#pragma unroll
        for (int i = 0; i < N; ++i) any0 |= w0[i], any1 |= w1[i];
        any0 &= drop;
        any1 &= drop;
      }
      if (next < p.M) {               // the next row is on its way while this one is worked on
        load16<T>(src + next * p.ldw, p.vec, in[0], w0);
        load16<T>(src + next * p.ldw + 64, p.vec, in[1], w1);
      }
      int e[2] = {-127, -127};
      bool finite[2] = {true, true};
      uint32_t c[2][2] = {{0u, 0u}, {0u, 0u}};
      if (PREP) {
        // sum of v^2 over the group's block (the group itself for smaller blocks); 0: nothing but zeros
        float2 q = make_float2(any0 ? 0x1p-120f : 0.0f, any1 ? 0x1p-120f : 0.0f);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[j] = mul2(x[j], factor(f, lane, j));
          q = fma2(x[j], x[j], q);
        }
        q = add2(q, make_float2(__shfl_xor_sync(0xffffffffu, q.x, 1), __shfl_xor_sync(0xffffffffu, q.y, 1)));
        if (LB > 5) q = add2(q, make_float2(__shfl_xor_sync(0xffffffffu, q.x, 2), __shfl_xor_sync(0xffffffffu, q.y, 2)));
        if (LB > 6) q.x = q.y = q.x + q.y;
#pragma unroll
        for (int t = 7; t < LB; ++t) q.x = q.y = q.x + __shfl_xor_sync(0xffffffffu, q.x, 1 << (t - 5));
        rotate<LB>(x, lane);
        float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          top = make_float2(max_abs(top.x, x[j].x, x[j + 1].x), max_abs(top.y, x[j].y, x[j + 1].y));
        top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, 1));
        top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, 1));
        constexpr float kBound = (float)(LB + 6) * 0x1p-24f;
        constexpr float kTerms = (float)(1 << (LB > 5 ? LB : 5));
        float2 scale, ms;             // 2^-e / sqrt(b) and m 2^-e of each run
        uint32_t again[2] = {0u, 0u}; // the run's values to be decided from fp64
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float Q = r ? q.y : q.x, t = (r ? top.y : top.x) * inv;
          const float m = kBound * inv * sqrtf(kTerms * Q);
          const float lo = fmaxf(t - m, 0.0f), hi = t + m;
          e[r] = (int)(__float_as_uint(lo) >> 23) - 127 - 2;
          const bool zero = Q == 0.0f || !in[r];
          // The third condition: a group that cancels to within some times m. It leaves 2 m 2^-e <= 1/4, so that
          // y - m and y + m, where they differ in sign, both round to 0: |y +- m| is then at most 2 m.
          const bool sure = Q > 0x1p-100f && Q < 0x1p100f && 64.0f * m <= lo &&
                            (__float_as_uint(lo) >> 23) == (__float_as_uint(hi) >> 23);
          if (!sure) e[r] = -127;
          if (!sure && !zero) again[r] = 0xffffu;
          const float up = sure ? __uint_as_float((uint32_t)(127 - e[r]) << 23) : 0.0f;   // !sure: codes 0 for now
          (r ? scale.y : scale.x) = inv * up;
          (r ? ms.y : ms.x) = sure ? m * up : 0.0f;
        }
        const float2 less = make_float2(-ms.x, -ms.y);
        float u[2][16], v[2][16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 a = fma2(x[j], scale, less), b = fma2(x[j], scale, ms);
          u[0][j] = a.x, u[1][j] = a.y, v[0][j] = b.x, v[1][j] = b.y;
        }
        uint32_t open = again[0] | again[1];
        uint32_t d[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = e2m1x8(u[r] + 8 * h), b = e2m1x8(v[r] + 8 * h);
            c[r][h] = a & b;          // a difference in the sign alone: both are 0 (see `sure`), and so is the value
            d[r][h] = (a ^ b) & 0x77777777u;
            open |= d[r][h];
          }
        }
        if (__any_sync(0xffffffffu, open != 0u)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if ((d[r][i >> 3] >> (4 * (i & 7))) & 15u) again[r] |= 1u << i;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, again[r], 1);
            const uint32_t all = (lane & 1) ? (other | (again[r] << 16)) : (again[r] | (other << 16));
            for (uint32_t lanes = __ballot_sync(0xffffffffu, all != 0u) & 0x55555555u; lanes != 0u;
                 lanes &= lanes - 1u) {
              const int l = __ffs((int)lanes) - 1;
              const Decided n = decide_exactly<T>(p, row, __shfl_sync(0xffffffffu, at.group0, l) + 2 * r,
                                                  __shfl_sync(0xffffffffu, all, l), __shfl_sync(0xffffffffu, e[r], l));
              if ((lane & ~1) == l) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t code = (lane & 1) ? n.code[2 + h] : n.code[h];
                  const uint32_t mask = (lane & 1) ? n.mask[2 + h] : n.mask[h];
                  c[r][h] = (c[r][h] & ~mask) | code;
                }
                e[r] = n.e;
                finite[r] = n.finite;
              }
            }
          }
        }
      } else {
        uint32_t top[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          top[0] = max(top[0], __float_as_uint(x[j].x) & 0x7FFFFFFFu);
          top[1] = max(top[1], __float_as_uint(x[j].y) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = max(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          finite[r] = top[r] < 0x7F800000u;
          e[r] = max((int)(top[r] >> 23) - 127 - 2, -127);   // a subnormal maximum: -127
          // 2^-e is a normal float for every e in -127 .. 125
          const float up = __uint_as_float((uint32_t)(127 - e[r]) << 23);
          float u[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) u[j] = __fmul_rn(r ? x[j].y : x[j].x, up);
          c[r][0] = e2m1x8(u);
          c[r][1] = e2m1x8(u + 8);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (in[r]) {
          if (!finite[r]) {
            c[r][0] = c[r][1] = 0u;
            bad |= QAMW_STATUS_NONFINITE_INPUT;
          }
          // the two groups of this lane's scale word: bytes (lane bit 1) and 2 + (lane bit 1)
          sword |= (finite[r] ? (uint32_t)(e[r] + 127) : 255u) << (16 * r + 4 * (lane & 2));
          *reinterpret_cast<uint2 *>(p.codes + row * (p.K / 2) + at.run0 / 2 + 32 * r) = make_uint2(c[r][0], c[r][1]);
        }
      }
    }
    sword |= __shfl_xor_sync(0xffffffffu, sword, 2);
    if ((lane & 3) == 0 && at.group0 / 4 < k_tiles)
      *reinterpret_cast<uint32_t *>(p.scales + scale_offset(row, at.group0, k_tiles)) = sword;
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) status_or(p.status, bad);
}

struct MxDecodeArgs {
  const uint8_t *codes, *scales;
  int64_t M, K;
  const float *s;       // [K] or nullptr
  int divide;           // the quantisation divided by s: multiply here
  int log2b;
  uint64_t seed;
  void *out;
  int64_t ldo;
  int64_t units_k, row_groups;
  int vec;
};

// 16 columns of a run
__device__ __forceinline__ void store16(float *p, int vec, const float (&x)[16]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[8 * i + j]);
      store_32b(p + 8 * i, vec, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) p[j] = x[j];
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, int vec, const float (&x)[16]) {
  if (vec) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    store_32b(p, vec, w);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) p[j] = __float2bfloat16_rn(x[j]);
  }
}

// Scale bytes from which the decode's fp32 sums (of up to 32 groups, each up to
// 32 x 6 x 2^e) may overflow: e > 112. Small ones lose nothing: the sums are
// multiples of 2^-128, which fp32 holds down to its subnormal numbers.
constexpr uint32_t kBeyondFp32 = 240;

// The rows of a warp that have such a byte (found by one more pass over their
// scales), or all of them if a column's factor is no normal number, from the
// definition, in fp64 and rounded once: a value may be within the type although
// the sum before its division by sqrt(b) s is not, or the other way round.
template <typename T>
__device__ __noinline__ void decode_exactly(const MxDecodeArgs &p, bool every) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x % p.units_k, first = (blockIdx.x / p.units_k) * kMxWarps + (threadIdx.x >> 5);
  const int64_t k_tiles = (p.K + 127) / 128, run0 = LanePlace(unit, lane).run0, b = (int64_t)1 << p.log2b;
  const int64_t end = min((unit + 1) * kMxUnit, p.K);
  __syncwarp();                       // the lanes' stores of the pass before come first
  for (int64_t row = first; row < p.M; row += p.row_groups) {
    const uint8_t *codes = p.codes + row * (p.K / 2);
    bool beyond = every;
    for (int64_t c = run0; c < run0 + 128 && c < p.K; c += 64)
      beyond |= p.scales[scale_offset(row, c / 32, k_tiles)] >= kBeyondFp32;
    if (!__any_sync(0xffffffffu, beyond)) continue;
    for (int64_t col = unit * kMxUnit + lane; col < end; col += 32) {
      double x = 0.0;
      for (int64_t c = col & ~(b - 1), last = c + b; c < last; ++c) {
        const uint32_t byte = p.scales[scale_offset(row, c / 32, k_tiles)], q = codes[c / 2] >> (4 * (c & 1));
        double v = (double)((0xC8643210u >> (4 * (q & 7u))) & 15u);               // twice the element
        v *= byte == 255u ? nan("") : __hiloint2double((int)(byte + 895u) << 20, 0);   // 2^(byte - 128)
        x += ((q >> 3) ^ __popcll(c & col & (b - 1))) & 1 ? -v : v;
      }
      if (p.log2b > 0) x *= (mask_is_negative(p.seed, col) ? -1.0 : 1.0) / sqrt((double)b);
      if (p.s != nullptr) x = p.divide ? x * (double)p.s[col] : x / (double)p.s[col];
      T *o = static_cast<T *>(p.out) + row * p.ldo + col;
      if constexpr (sizeof(T) == 2) *o = __double2bfloat16(x);
      else *o = (float)x;
    }
  }
}

// x = d (.) (H_b q 2^e) / (sqrt(b) s) (times s for divided rows): one rounding
// to the output type at the end, like the codec's own decode; without a
// rotation and a scale every value is exact in either type. Lanes hold what
// they hold in the quantisation. Block bits 0-4 stay inside a group, whose
// values share a scale: their sums (at most 32 x 6, in halves) are exact in
// fp16, two columns an instruction and two an exchange between lanes. Then the
// scale, and the other bits in fp32. 11008 x 4096 bf16 at b = 128: 33 us (3.5
// TB/s), 5120 x 13824 at b = 256: 52 us (with all bits in fp32 and the factors in
// shared memory 59, its L1 pipe 81% busy; now 62%, at b = 128 49%). No pipe is
// full: 13 warps per SM issue in 57-60% of the slots, and wait for fixed
// latencies and for the next row's loads.
template <typename T, int LB>
__global__ void __launch_bounds__(32 * kMxWarps, (LB > 0 ? kMxResident : kMxResidentPlain) / kMxWarps)
    mx4_decode_kernel(const __grid_constant__ MxDecodeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = blockIdx.x % p.units_k, rg = (blockIdx.x / p.units_k) * kMxWarps + (threadIdx.x >> 5);
  const LanePlace at(unit, lane);
  const int64_t k_tiles = (p.K + 127) / 128;
  const bool in0 = at.run0 < p.K, in1 = at.run0 + 64 < p.K;
  uint2 c0 = make_uint2(0u, 0u), c1 = make_uint2(0u, 0u);
  uint32_t sw = 0;                    // the scale bytes of four groups, two of them this lane's
  auto fetch = [&](int64_t row) {
    const uint8_t *q = p.codes + row * (p.K / 2) + at.run0 / 2;
    if (in0) {
      c0 = *reinterpret_cast<const uint2 *>(q);
      sw = *reinterpret_cast<const uint32_t *>(p.scales + scale_offset(row, at.group0 & ~(int64_t)3, k_tiles));
    }
    if (in1) c1 = *reinterpret_cast<const uint2 *>(q + 32);
  };
  if (rg < p.M) fetch(rg);
  const float inv = (float)(1.0 / sqrt((double)(1 << LB)));
  __shared__ Factors shared;
  bool odd = false;                   // a factor that is no normal number
  form_factors(shared, unit, p.K, [&](int64_t col) {
    float v = inv;
    if (p.s != nullptr) v = p.divide ? __fmul_rn(inv, p.s[col]) : __fdiv_rn(inv, p.s[col]);
    odd |= !(fabsf(v) >= 0x1p-126f && fabsf(v) < INFINITY);
    return (LB > 0 && mask_is_negative(p.seed, col)) ? -v : v;
  });
  float2 f[LB > 0 ? 16 : 1];          // in registers where the exchanges keep the L1 pipe busy
  if constexpr (LB > 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = factor(shared, lane, j);
  }
  uint32_t top = __syncthreads_or(odd) ? 256u : 0u;   // the largest scale byte, or 256
  for (int64_t row = rg; row < p.M; row += p.row_groups) {
    __half2 h[16];                    // (run 0, run 1) of column j
    {
      uint32_t a[8], b[8];
      halves_of_e2m1x8(c0.x, a);
      halves_of_e2m1x8(c0.y, a + 4);
      halves_of_e2m1x8(c1.x, b);
      halves_of_e2m1x8(c1.y, b + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t lo = __byte_perm(a[i], b[i], 0x5410), hi = __byte_perm(a[i], b[i], 0x7632);
        h[2 * i] = *reinterpret_cast<const __half2 *>(&lo);
        h[2 * i + 1] = *reinterpret_cast<const __half2 *>(&hi);
      }
    }
    const uint32_t sh = 4 * (lane & 2);
    const uint32_t b0 = (sw >> sh) & 255u, b1 = (sw >> (16 + sh)) & 255u;
    const float2 g = make_float2(e8m0_value(b0), e8m0_value(b1));
    top = max(top, max(b0, b1));
    if (row + p.row_groups < p.M) fetch(row + p.row_groups);
#pragma unroll
    for (int t = 0; t < (LB < 4 ? LB : 4); ++t) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if ((j & (1 << t)) == 0) {
          const __half2 a = h[j], b = h[j | (1 << t)];
          h[j] = __hadd2(a, b);
          h[j | (1 << t)] = __hsub2(a, b);
        }
      }
    }
    if constexpr (LB > 4) {
      const __half2 s = __float2half2_rn((lane & 1) ? -1.0f : 1.0f);
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = __hfma2(h[j], s, __shfl_xor_sync(0xffffffffu, h[j], 1));
    }
    float2 x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = mul2(__half22float2(h[j]), g);
    if constexpr (LB > 6) butterflies_pair(x);
    if constexpr (LB > 5) butterflies_lane(x, lane, 2);
#pragma unroll
    for (int t = 7; t < LB; ++t) butterflies_lane(x, lane, 1 << (t - 5));
    float u[16], v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 y = mul2(x[j], LB > 0 ? f[LB > 0 ? j : 0] : factor(shared, lane, j));
      u[j] = y.x;
      v[j] = y.y;
    }
    T *o = static_cast<T *>(p.out) + row * p.ldo + at.run0;
    if (in0) store16(o, p.vec, u);
    if (in1) store16(o + 64, p.vec, v);
  }
  // without a rotation and a scale the values are exact for every byte
  if ((LB > 0 || p.s != nullptr) && __any_sync(0xffffffffu, top >= kBeyondFp32)) decode_exactly<T>(p, top == 256u);
}

// One scale byte per (row, group), row-major, into the tiled layout (or back);
// the padding of the tiles is written as 0.
__global__ void mx4_scale_layout_kernel(const uint8_t *in, uint8_t *out, int64_t M, int64_t groups, int64_t k_tiles,
                                        int64_t n, int to_tiles) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t per_row = k_tiles * 4, row = i / per_row, g = i % per_row;
    const int64_t t = scale_offset(row, g, k_tiles);
    const bool real = row < M && g < groups;
    if (to_tiles) out[t] = real ? in[row * groups + g] : (uint8_t)0;
    else if (real) out[row * groups + g] = in[t];
  }
}

// Rows of one column unit are dealt out to as many warps as the GPU holds at
// once (`resident` per SM), so that there is one wave and the column factors
// are formed once for all rows of a CTA.
int64_t row_groups_for(int64_t rows, int64_t units_k, int resident) {
  const int64_t ctas = (int64_t)sm_count() * (resident / kMxWarps) / units_k, most = (rows + kMxWarps - 1) / kMxWarps;
  return kMxWarps * (ctas < 1 ? 1 : ctas < most ? ctas : most);
}

// Calls f with log2 b as a compile-time constant: the butterflies of a block
// are then straight code (every block size has its kernel).
template <typename F>
void with_log2b(int log2b, F f) {
  switch (log2b) {
    case 0: return f(std::integral_constant<int, 0>());
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    case 8: return f(std::integral_constant<int, 8>());
    case 9: return f(std::integral_constant<int, 9>());
    default: return f(std::integral_constant<int, 10>());
  }
}

// the widest vector access (32, 16 or 0 bytes) that every row allows
int vector_bytes(const void *p, int64_t pitch) {
  const uint64_t a = reinterpret_cast<uintptr_t>(p) | (uint64_t)pitch;
  return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 0;
}

}  // namespace

cudaError_t launch_mx4_quantize(const Mx4QuantizeArgs &a, cudaStream_t s) {
  MxQuantArgs p;
  p.W = a.W;
  p.M = a.M;
  p.K = a.K;
  p.ldw = a.ldw;
  p.s = a.col_scale;
  p.divide = a.divide;
  p.log2b = a.log2b;
  p.seed = a.seed;
  p.codes = a.codes;
  p.scales = a.scales;
  p.status = a.status;
  p.units_k = (a.K + kMxUnit - 1) / kMxUnit;
  const int es = a.wt == QAMW_BF16 ? 2 : 4;
  p.vec = vector_bytes(a.W, a.ldw * es);
  const bool plain = a.col_scale == nullptr && a.log2b == 0;
  p.row_groups = row_groups_for((a.M + 127) / 128 * 128, p.units_k, plain ? kMxResidentPlain : kMxResident);
  const dim3 grid((unsigned)(p.units_k * (p.row_groups / kMxWarps)));
  auto run = [&](auto kernel) { kernel<<<grid, 32 * kMxWarps, 0, s>>>(p); };
  if (plain) {
    if (a.wt == QAMW_BF16) run(mx4_quantize_kernel<uint16_t, false, 0>);
    else run(mx4_quantize_kernel<float, false, 0>);
  } else {
    with_log2b(a.log2b, [&](auto lb) {
      if (a.wt == QAMW_BF16) run(mx4_quantize_kernel<uint16_t, true, decltype(lb)::value>);
      else run(mx4_quantize_kernel<float, true, decltype(lb)::value>);
    });
  }
  return cudaGetLastError();
}

cudaError_t launch_mx4_decode(const Mx4DecodeArgs &a, cudaStream_t s) {
  MxDecodeArgs p;
  p.codes = a.codes;
  p.scales = a.scales;
  p.M = a.M;
  p.K = a.K;
  p.s = a.col_scale;
  p.divide = a.divide;
  p.log2b = a.log2b;
  p.seed = a.seed;
  p.out = a.out;
  p.ldo = a.ldo;
  p.units_k = (a.K + kMxUnit - 1) / kMxUnit;
  const int es = a.out_t == QAMW_BF16 ? 2 : 4;
  p.vec = vector_bytes(a.out, a.ldo * es);
  p.row_groups = row_groups_for(a.M, p.units_k, a.log2b > 0 ? kMxResident : kMxResidentPlain);
  const dim3 grid((unsigned)(p.units_k * (p.row_groups / kMxWarps)));
  with_log2b(a.log2b, [&](auto lb) {
    if (a.out_t == QAMW_BF16) mx4_decode_kernel<__nv_bfloat16, decltype(lb)::value><<<grid, 32 * kMxWarps, 0, s>>>(p);
    else mx4_decode_kernel<float, decltype(lb)::value><<<grid, 32 * kMxWarps, 0, s>>>(p);
  });
  return cudaGetLastError();
}

cudaError_t launch_mx4_scale_layout(const uint8_t *in, uint8_t *out, int64_t M, int64_t K, bool to_tiles,
                                    cudaStream_t s) {
  const int64_t k_tiles = (K + 127) / 128, rows = to_tiles ? (M + 127) / 128 * 128 : M;
  const int64_t n = rows * k_tiles * 4;
  const int64_t blocks = (n + 255) / 256, most = (int64_t)sm_count() * 16;
  mx4_scale_layout_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, s>>>(in, out, M, K / 32, k_tiles, n,
                                                                                    to_tiles ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace qamw
