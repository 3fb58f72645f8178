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
// differ (about 2 in 10^5 values of Gaussian rows at b = 128), or the group's
// exponent hangs on the error, the warp forms the value in fp64 from the row.
// An e2m1 border has at most three significant bits, so the exponent and the
// top mantissa bits of that double, with a sticky bit for the rest, decide
// exactly (double_scaled).
//
// Error of the fp32 value, with A = sum of |v| over the block: v itself 2 x
// 2^-24 (1/s rounded, and the product), one rounding of at most 2^-24 A per
// butterfly level, the factor 2^-e / sqrt(b) and its product 2 x 2^-24, and the
// sum y +- m one more: (log2 b + 6) 2^-24 A, with one 2^-24 A for the error of A.
//
// A lane loads two runs of 16 columns, 64 columns apart, so that four lanes
// read 128 contiguous bytes of bf16; block bits 0-3 and 6 are butterflies on
// its registers. An exchange of half the registers with the neighbour lane
// swaps column bits 4 and 6: then the lane holds one whole group of 32 columns,
// bit 4 is a register butterfly too, the group's maximum needs no exchange and
// its codes are one 16-byte store. Bit 5 and bits 7-9 are lane exchanges.
#include <cuda_fp16.h>

#include "qamw_device.cuh"
#include "qamw_internal.h"

namespace qamw {
namespace {

constexpr int kMxWarps = 8;         // warps per CTA
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
// eight e2m1 codes -> floats
__device__ __forceinline__ void floats_of_e2m1x8(uint32_t w, float *v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
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

// one fp64 value of the prepared row: y_col = sum_i (-1)^popc(i & col) d_i v_i / sqrt(b)
// over the columns i of its block, formed by the whole warp
template <typename T>
__device__ __noinline__ double exact_value(const MxQuantArgs &p, int64_t row, int64_t col) {
  const int lane = threadIdx.x & 31, b = 1 << p.log2b;
  const int64_t base = col & ~(int64_t)(b - 1);
  const void *w = static_cast<const T *>(p.W) + row * p.ldw;
  double y = 0.0;
  for (int i = lane; i < b; i += 32) {
    const int64_t c = base + i;
    double v = Raw<T>::exact(w, c);
    if (p.s != nullptr) v = p.divide ? v / (double)p.s[c] : v * (double)p.s[c];
    if (p.log2b > 0 && (mask_is_negative(p.seed, c) != ((__popc(i & (int)(col - base)) & 1) != 0))) v = -v;
    y += v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
  return p.log2b > 0 ? y * (1.0 / sqrt((double)b)) : y;
}

// Decides the values of `mask` of lane `src`'s group again, from fp64; with
// all of them (mask ~0) the group's exponent too. Warp-collective.
template <typename T>
__device__ __noinline__ void decide_exactly(const MxQuantArgs &p, int64_t row, int64_t group, uint32_t mask, int src,
                                            int &e, uint4 &codes, bool &finite) {
  const int lane = threadIdx.x & 31;
  double mine = 0.0;
  for (uint32_t left = mask; left != 0u; left &= left - 1u) {
    const int k = __ffs((int)left) - 1;
    const double y = exact_value<T>(p, row, 32 * group + k);
    if (lane == k) mine = y;
  }
  int ex = __shfl_sync(0xffffffffu, e, src);
  bool fin = true;
  if (mask == 0xffffffffu) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, (uint32_t)__double2hiint(mine) & 0x7FFFFFFFu);
    fin = top < 0x7FF00000u;
    ex = min(max((int)(top >> 20) - 1023 - 2, -127), 127);
  }
  const float pair[8] = {fin ? double_scaled(mine, ex) : 0.0f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool own = (mask >> lane) & 1u;
  uint32_t n = own ? (e2m1x8(pair) & 15u) << (4 * (lane & 7)) : 0u;     // this value's code, in its place
  uint32_t m = own ? 15u << (4 * (lane & 7)) : 0u;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    n |= __shfl_xor_sync(0xffffffffu, n, o);
    m |= __shfl_xor_sync(0xffffffffu, m, o);
  }
  uint32_t nw[4], mw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    nw[i] = __shfl_sync(0xffffffffu, n, 8 * i);
    mw[i] = __shfl_sync(0xffffffffu, m, 8 * i);
  }
  if (lane == src) {
    codes.x = (codes.x & ~mw[0]) | nw[0];
    codes.y = (codes.y & ~mw[1]) | nw[1];
    codes.z = (codes.z & ~mw[2]) | nw[2];
    codes.w = (codes.w & ~mw[3]) | nw[3];
    e = ex;
    finite = fin;
  }
}

// The lane's place in a unit of 1024 columns: column bits 4 and 5 of its loads
// are lane bits 0 and 1, bit 6 its two runs, bits 7-9 lane bits 2-4.
struct LanePlace {
  int64_t run0;    // first column of run 0; run 1 starts 64 columns on
  int64_t group;   // the group that it holds after the exchange
  int sub;         // that group's place among the four of its scale word
  __device__ __forceinline__ LanePlace(int64_t unit, int lane) {
    const int64_t sb = unit * kMxUnit + 128 * (lane >> 2);
    run0 = sb + 32 * ((lane >> 1) & 1) + 16 * (lane & 1);
    sub = 2 * (lane & 1) + ((lane >> 1) & 1);
    group = sb / 32 + sub;
  }
};

// x[j] = (run 0, run 1) of column j  ->  y[j] = columns (j, j + 16) of the
// lane's group (to_group), or back: lane bit 0 and the run trade places.
__device__ __forceinline__ void exchange(float2 (&x)[16], int lane) {
  const bool odd = (lane & 1) != 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? x[j].x : x[j].y, 1);
    if (odd) x[j].x = got;
    else x[j].y = got;
  }
}

__device__ __forceinline__ float2 diff2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }

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

// Signed column factors of the lane's 2 x 16 loaded columns: +-s, +-1/s or +-1.
// A factor far from 1 becomes NaN: its rows are then decided from fp64.
__device__ __forceinline__ void column_factors(const float *s, int divide, int log2b, uint64_t seed, int64_t run0,
                                               int64_t K, float2 (&f)[16]) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t col = run0 + 64 * c + j;
      float v = 1.0f;
      if (col < K) {
        if (s != nullptr) {
          v = divide ? __frcp_rn(s[col]) : s[col];
          if (!(fabsf(v) > 0x1p-100f && fabsf(v) < 0x1p100f)) v = __uint_as_float(0x7FC00000u);
        }
        if (log2b > 0 && mask_is_negative(seed, col)) v = -v;
      }
      if (c == 0) f[j].x = v;
      else f[j].y = v;
    }
  }
}

// PREP: a channel scale or a rotation; otherwise the values are exact as read.
template <typename T, bool PREP>
__global__ void __launch_bounds__(32 * kMxWarps) mx4_quantize_kernel(MxQuantArgs p) {
  constexpr int N = Raw<T>::kWords;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5);
  if (id >= p.units_k * p.row_groups) return;
  const int64_t unit = id % p.units_k, rg = id / p.units_k;
  const LanePlace at(unit, lane);
  const int64_t k_tiles = (p.K + 127) / 128, rows_pad = (p.M + 127) / 128 * 128;
  // K % 32 == 0: a run of 16 columns and a group are all in or all out
  const bool in0 = at.run0 < p.K, in1 = at.run0 + 64 < p.K, in = 32 * at.group < p.K;
  const T *src = static_cast<const T *>(p.W) + at.run0;
  float2 f[16];
  if (PREP) column_factors(p.s, p.divide, p.log2b, p.seed, at.run0, p.K, f);
  const float inv = (float)(1.0 / sqrt((double)(1 << p.log2b)));
  const float bound = (float)(p.log2b + 7) * 0x1p-24f;
  uint32_t bad = 0;
  uint32_t w0[N], w1[N];
  if (rg < p.M) {
    load16<T>(src + rg * p.ldw, p.vec, in0, w0);
    load16<T>(src + rg * p.ldw + 64, p.vec, in1, w1);
  }
  for (int64_t row = rg; row < rows_pad; row += p.row_groups) {
    uint32_t sbyte = 0;
    if (row < p.M) {
      float2 x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = make_float2(Raw<T>::value(w0, j), Raw<T>::value(w1, j));
      uint32_t any0 = 0, any1 = 0;    // nonzero bits of each run, signs apart
      if (PREP) {
        const uint32_t drop = N == 8 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
#pragma unroll
        for (int i = 0; i < N; ++i) any0 |= w0[i] & drop, any1 |= w1[i] & drop;
      }
      const int64_t next = row + p.row_groups;
      if (next < p.M) {               // the next row is on its way while this one is worked on
        load16<T>(src + next * p.ldw, p.vec, in0, w0);
        load16<T>(src + next * p.ldw + 64, p.vec, in1, w1);
      }
      int e = -127;
      bool finite = true;
      uint4 c = make_uint4(0u, 0u, 0u, 0u);
      if (PREP) {
        float2 sum = make_float2(any0 ? 0x1p-120f : 0.0f, any1 ? 0x1p-120f : 0.0f);   // |v| of each run; 0: a run of zeros
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[j] = mul2(x[j], f[j]);
          sum = add2(sum, make_float2(fabsf(x[j].x), fabsf(x[j].y)));
        }
        // A over the group's block (the group itself for smaller blocks)
        const bool odd = (lane & 1) != 0;
        float A = (odd ? sum.y : sum.x) + __shfl_xor_sync(0xffffffffu, odd ? sum.x : sum.y, 1);
        if (p.log2b > 5) A += __shfl_xor_sync(0xffffffffu, A, 2);
        if (p.log2b > 6) A += __shfl_xor_sync(0xffffffffu, A, 1);
        for (int t = 7; t < p.log2b; ++t) A += __shfl_xor_sync(0xffffffffu, A, 1 << (t - 5));
        butterflies_low(x, p.log2b);
        if (p.log2b > 6) butterflies_pair(x);
        exchange(x, lane);
        if (p.log2b > 4) butterflies_pair(x);
        if (p.log2b > 5) butterflies_lane(x, lane, 2);
        for (int t = 7; t < p.log2b; ++t) butterflies_lane(x, lane, 1 << (t - 5));
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
        const float m = bound * A * inv;
        const float lo = fmaxf(top * inv - m, 0.0f), hi = top * inv + m;
        e = (int)(__float_as_uint(lo) >> 23) - 127 - 2;
        uint32_t again = 0;           // the group's values to be decided from fp64
        if (in && A != 0.0f) {
          const bool sure = A > 0x1p-90f && A < 0x1p90f && (__float_as_uint(lo) >> 23) == (__float_as_uint(hi) >> 23);
          if (sure) {
            const float scale = inv * __uint_as_float((uint32_t)(127 - e) << 23), ms = m * __uint_as_float((uint32_t)(127 - e) << 23);
            float u[16], v[16];
            uint32_t cw[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float t = h ? x[j].y : x[j].x;
                u[j] = __fmaf_rn(t, scale, -ms);
                v[j] = __fmaf_rn(t, scale, ms);
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t a = e2m1x8(u + 8 * q), b = e2m1x8(v + 8 * q);
                // a value within m of zero differs in its sign alone: it is +0
                cw[2 * h + q] = a & b;
                const uint32_t d = (a ^ b) & 0x77777777u;
                if (d != 0u) {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if ((d >> (4 * i)) & 15u) again |= 1u << (16 * h + 8 * q + i);
                }
              }
            }
            c = make_uint4(cw[0], cw[1], cw[2], cw[3]);
          } else {
            again = 0xffffffffu;
          }
        } else {
          e = -127;                   // nothing but zeros
        }
        for (uint32_t lanes = __ballot_sync(0xffffffffu, again != 0u); lanes != 0u; lanes &= lanes - 1u) {
          const int l = __ffs((int)lanes) - 1;
          decide_exactly<T>(p, row, __shfl_sync(0xffffffffu, at.group, l), __shfl_sync(0xffffffffu, again, l), l, e, c,
                            finite);
        }
      } else {
        exchange(x, lane);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          top = max(top, __float_as_uint(x[j].x) & 0x7FFFFFFFu);
          top = max(top, __float_as_uint(x[j].y) & 0x7FFFFFFFu);
        }
        finite = top < 0x7F800000u;
        e = max((int)(top >> 23) - 127 - 2, -127);   // a subnormal maximum: -127
        // 2^-e is a normal float for every e in -127 .. 125
        const float scale = __uint_as_float((uint32_t)(127 - e) << 23);
        float u[16], v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) u[j] = __fmul_rn(x[j].x, scale), v[j] = __fmul_rn(x[j].y, scale);
        c = make_uint4(e2m1x8(u), e2m1x8(u + 8), e2m1x8(v), e2m1x8(v + 8));
      }
      if (in) {
        if (!finite) {
          c = make_uint4(0u, 0u, 0u, 0u);
          bad |= QAMW_STATUS_NONFINITE_INPUT;
        }
        sbyte = finite ? (uint32_t)(e + 127) : 255u;
        *reinterpret_cast<uint4 *>(p.codes + row * (p.K / 2) + 16 * at.group) = c;
      }
    }
    // four lanes' scale bytes form one word of a tile
    uint32_t w = sbyte << (8 * at.sub);
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if ((lane & 3) == 0 && at.group / 4 < k_tiles)
      *reinterpret_cast<uint32_t *>(p.scales + scale_offset(row, at.group, k_tiles)) = w;
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

// x = d (.) (H_b q 2^e) / (sqrt(b) s) (times s for divided rows): fp32
// arithmetic, one rounding to the output type, like the codec's own decode.
// Without a rotation and a scale every value is exact in either type. The
// lane's group of 32 columns goes the quantisation's way back: pairs and lane
// exchanges, the exchange of runs, then the bits of a run, and the column
// factor d / (sqrt(b) s), formed once for all rows of the warp.
template <typename T>
__global__ void __launch_bounds__(32 * kMxWarps) mx4_decode_kernel(MxDecodeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5);
  if (id >= p.units_k * p.row_groups) return;
  const int64_t unit = id % p.units_k, rg = id / p.units_k;
  const LanePlace at(unit, lane);
  const int64_t k_tiles = (p.K + 127) / 128;
  const bool in0 = at.run0 < p.K, in1 = at.run0 + 64 < p.K, in = 32 * at.group < p.K;
  const float inv = (float)(1.0 / sqrt((double)(1 << p.log2b)));
  float2 f[16];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int64_t col = at.run0 + 64 * c + j;
      float v = inv;
      if (col < p.K) {
        if (p.s != nullptr) v = p.divide ? __fmul_rn(inv, p.s[col]) : __fdiv_rn(inv, p.s[col]);
        if (p.log2b > 0 && mask_is_negative(p.seed, col)) v = -v;
      }
      if (c == 0) f[j].x = v;
      else f[j].y = v;
    }
  }
  uint4 c = make_uint4(0u, 0u, 0u, 0u);
  uint32_t sb = 0;
  auto fetch = [&](int64_t row) {
    if (in) {
      c = *reinterpret_cast<const uint4 *>(p.codes + row * (p.K / 2) + 16 * at.group);
      sb = p.scales[scale_offset(row, at.group, k_tiles)];
    }
  };
  if (rg < p.M) fetch(rg);
  for (int64_t row = rg; row < p.M; row += p.row_groups) {
    float u[16], v[16];
    floats_of_e2m1x8(c.x, u);
    floats_of_e2m1x8(c.y, u + 8);
    floats_of_e2m1x8(c.z, v);
    floats_of_e2m1x8(c.w, v + 8);
    const float g = e8m0_value(sb);
    if (row + p.row_groups < p.M) fetch(row + p.row_groups);
    float2 x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = make_float2(__fmul_rn(u[j], g), __fmul_rn(v[j], g));
    for (int t = 7; t < p.log2b; ++t) butterflies_lane(x, lane, 1 << (t - 5));
    if (p.log2b > 5) butterflies_lane(x, lane, 2);
    if (p.log2b > 4) butterflies_pair(x);
    exchange(x, lane);
    if (p.log2b > 6) butterflies_pair(x);
    butterflies_low(x, p.log2b);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 y = mul2(x[j], f[j]);
      u[j] = y.x;
      v[j] = y.y;
    }
    T *o = static_cast<T *>(p.out) + row * p.ldo + at.run0;
    if (in0) store16(o, p.vec, u);
    if (in1) store16(o + 64, p.vec, v);
  }
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

// Rows of one column unit are dealt out so that each warp has up to 16 rows
// (the sign mask of its columns is formed once for all of them), as long as
// enough warps remain to fill the GPU.
int64_t row_groups_for(int64_t rows, int64_t units_k) {
  const int64_t want = (int64_t)sm_count() * 16;            // warps that keep an SM busy
  int64_t per = rows * units_k / want;
  per = per < 1 ? 1 : per > 16 ? 16 : per;
  return (rows + per - 1) / per;
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
  p.row_groups = row_groups_for((a.M + 127) / 128 * 128, p.units_k);
  const int64_t warps = p.units_k * p.row_groups;
  const dim3 grid((unsigned)((warps + kMxWarps - 1) / kMxWarps));
  const bool prep = a.col_scale != nullptr || a.log2b > 0;
  if (a.wt == QAMW_BF16) {
    if (prep) mx4_quantize_kernel<uint16_t, true><<<grid, 32 * kMxWarps, 0, s>>>(p);
    else mx4_quantize_kernel<uint16_t, false><<<grid, 32 * kMxWarps, 0, s>>>(p);
  } else {
    if (prep) mx4_quantize_kernel<float, true><<<grid, 32 * kMxWarps, 0, s>>>(p);
    else mx4_quantize_kernel<float, false><<<grid, 32 * kMxWarps, 0, s>>>(p);
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
  p.row_groups = row_groups_for(a.M, p.units_k);
  const int64_t warps = p.units_k * p.row_groups;
  const dim3 grid((unsigned)((warps + kMxWarps - 1) / kMxWarps));
  if (a.out_t == QAMW_BF16) mx4_decode_kernel<__nv_bfloat16><<<grid, 32 * kMxWarps, 0, s>>>(p);
  else mx4_decode_kernel<float><<<grid, 32 * kMxWarps, 0, s>>>(p);
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
