// qamw_mx4.cu -- microscaled 4-bit floating point (OCP MX: e2m1 elements, one
// power-of-two scale per 32 columns): quantisation and decode, after the
// codec's own preparation of a row (Methodology (5) Activation-Aware Scaling
// and (2) Deterministic Rotation).
//
//   v_j = w_j s_j  or  w_j / s_j;   y = H_b (d (.) v) / sqrt(b)  per block of b columns
//   e   = clamp(floor(log2 max|y|) - 2, -127, 127) per group of 32 columns
//   q_j = the e2m1 value nearest y_j 2^-e (ties to the even code, at most 6)
//
// Rotation and scaling run in fp64 and no rounding lies between them and the
// 4-bit decision: an e2m1 border has at most three significant bits, so the
// exponent and the top mantissa bits of the double, with a sticky bit for the
// rest, decide exactly (double_scaled). One lane holds one group of 32
// consecutive columns: block bits 0-4 of the Hadamard transform are register
// butterflies, bits 5-9 exchanges between lanes, and the group's maximum needs
// no exchange at all.
#include <cuda_fp16.h>

#include "qamw_device.cuh"
#include "qamw_internal.h"

namespace qamw {
namespace {

constexpr int kMxWarps = 8;         // warps per CTA
constexpr int kMxUnit = 1024;       // columns per warp pass: 32 lanes x one group

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
  int vec;              // 16-byte loads allowed
};

template <typename T>
__device__ __forceinline__ void load32(const T *p, bool vec, float (&x)[32]);
template <>
__device__ __forceinline__ void load32<float>(const float *p, bool vec, float (&x)[32]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 q = reinterpret_cast<const float4 *>(p)[i];
      x[4 * i] = q.x, x[4 * i + 1] = q.y, x[4 * i + 2] = q.z, x[4 * i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = p[i];
  }
}
template <>
__device__ __forceinline__ void load32<uint16_t>(const uint16_t *p, bool vec, float (&x)[32]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4 *>(p)[i];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float((uint32_t)p[i] << 16);
  }
}

// the sign mask of the lane's 32 columns, bit j = column c0 + j negative
__device__ __forceinline__ uint32_t sign_bits(uint64_t seed, int64_t c0) {
  uint32_t m = 0;
#pragma unroll 4
  for (int j = 0; j < 32; ++j) m |= (uint32_t)(splitmix64_output(seed, (uint64_t)(c0 + j) + 1ull) >> 63) << j;
  return m;
}

// FP64: a channel scale or a rotation; otherwise the values are fp32 as read.
template <typename T, bool FP64>
__global__ void __launch_bounds__(32 * kMxWarps) mx4_quantize_kernel(MxQuantArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5);
  if (id >= p.units_k * p.row_groups) return;
  const int64_t unit = id % p.units_k, rg = id / p.units_k;
  const int64_t c0 = unit * kMxUnit + 32 * lane;
  const int64_t k_tiles = (p.K + 127) / 128, rows_pad = (p.M + 127) / 128 * 128;
  const bool in = c0 < p.K;            // K % 32 == 0: a lane's group is all in or all out
  const uint32_t neg = (FP64 && p.log2b > 0 && in) ? sign_bits(p.seed, c0) : 0u;
  const double inv_sqrt_b = FP64 ? 1.0 / sqrt((double)(1 << p.log2b)) : 1.0;
  uint32_t bad = 0;
  for (int64_t row = rg; row < rows_pad; row += p.row_groups) {
    uint32_t sbyte = 0;
    if (row < p.M) {
      float x[32];
      if (in) {
        load32<T>(static_cast<const T *>(p.W) + row * p.ldw + c0, p.vec != 0, x);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0.0f;
      }
      int e;
      bool finite;
      if (FP64) {
        double y[32];
        if (p.s != nullptr && in) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const double sj = (double)p.s[c0 + j];
            y[j] = p.divide ? (double)x[j] / sj : (double)x[j] * sj;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = (double)x[j];
        }
        if (p.log2b > 0) {
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] = ((neg >> j) & 1u) ? -y[j] : y[j];
#pragma unroll
          for (int t = 0; t < 5; ++t) {
            if (t < p.log2b) {
              const int h = 1 << t;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                if ((j & h) == 0) {
                  const double a = y[j], b = y[j | h];
                  y[j] = a + b;
                  y[j | h] = a - b;
                }
              }
            }
          }
          for (int t = 5; t < p.log2b; ++t) {
            const int h = 1 << (t - 5);
            const bool up = (lane & h) != 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const double o = __shfl_xor_sync(0xffffffffu, y[j], h);
              y[j] = up ? o - y[j] : y[j] + o;
            }
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j] *= inv_sqrt_b;
        }
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint32_t hi = (uint32_t)__double2hiint(y[j]) & 0x7FFFFFFFu;
          top = hi > top ? hi : top;
        }
        finite = top < 0x7FF00000u;
        e = max((int)(top >> 20) - 1023 - 2, -127);
        e = min(e, 127);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = double_scaled(y[j], e);
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint32_t u = __float_as_uint(x[j]) & 0x7FFFFFFFu;
          top = u > top ? u : top;
        }
        finite = top < 0x7F800000u;
        e = max((int)(top >> 23) - 127 - 2, -127);   // a subnormal maximum: -127
        // 2^-e is a normal float for every e in -127 .. 125
        const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __fmul_rn(x[j], f);
      }
      if (in) {
        uint4 c = make_uint4(0u, 0u, 0u, 0u);
        if (finite) c = make_uint4(e2m1x8(x), e2m1x8(x + 8), e2m1x8(x + 16), e2m1x8(x + 24));
        else bad |= QAMW_STATUS_NONFINITE_INPUT;
        sbyte = finite ? (uint32_t)(e + 127) : 255u;
        *reinterpret_cast<uint4 *>(p.codes + row * (p.K / 2) + c0 / 2) = c;
      }
    }
    // four lanes' scale bytes form one word of a tile
    uint32_t w = sbyte << (8 * (lane & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if ((lane & 3) == 0 && c0 / 128 < k_tiles)
      *reinterpret_cast<uint32_t *>(p.scales + scale_offset(row, c0 / 32, k_tiles)) = w;
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

__device__ __forceinline__ void store32(float *p, bool vec, const float (&x)[32]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) p[i] = x[i];
  }
}
__device__ __forceinline__ void store32(__nv_bfloat16 *p, bool vec, const float (&x)[32]) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 h[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
      reinterpret_cast<uint4 *>(p)[i] = *reinterpret_cast<const uint4 *>(h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) p[i] = __float2bfloat16_rn(x[i]);
  }
}

// x = d (.) (H_b q 2^e) / sqrt(b), divided by s (or times s): fp32 arithmetic,
// one rounding to the output type, like the codec's own decode. Without a
// rotation and a scale every value is exact in either type.
template <typename T>
__global__ void __launch_bounds__(32 * kMxWarps) mx4_decode_kernel(MxDecodeArgs p) {
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5);
  if (id >= p.units_k * p.row_groups) return;
  const int64_t unit = id % p.units_k, rg = id / p.units_k;
  const int64_t c0 = unit * kMxUnit + 32 * lane;
  const int64_t k_tiles = (p.K + 127) / 128;
  const bool in = c0 < p.K;
  const uint32_t neg = (p.log2b > 0 && in) ? sign_bits(p.seed, c0) : 0u;
  const float inv_sqrt_b = (float)(1.0 / sqrt((double)(1 << p.log2b)));
  for (int64_t row = rg; row < p.M; row += p.row_groups) {
    float x[32];
    if (in) {
      const uint4 c = *reinterpret_cast<const uint4 *>(p.codes + row * (p.K / 2) + c0 / 2);
      const float f = e8m0_value(p.scales[scale_offset(row, c0 / 32, k_tiles)]);
      floats_of_e2m1x8(c.x, x);
      floats_of_e2m1x8(c.y, x + 8);
      floats_of_e2m1x8(c.z, x + 16);
      floats_of_e2m1x8(c.w, x + 24);
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = __fmul_rn(x[j], f);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = 0.0f;
    }
    if (p.log2b > 0) {
#pragma unroll
      for (int t = 0; t < 5; ++t) {
        if (t < p.log2b) {
          const int h = 1 << t;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if ((j & h) == 0) {
              const float a = x[j], b = x[j | h];
              x[j] = a + b;
              x[j | h] = a - b;
            }
          }
        }
      }
      for (int t = 5; t < p.log2b; ++t) {
        const int h = 1 << (t - 5);
        const float sgn = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __fmaf_rn(sgn, x[j], __shfl_xor_sync(0xffffffffu, x[j], h));
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) x[j] = __fmul_rn(x[j], ((neg >> j) & 1u) ? -inv_sqrt_b : inv_sqrt_b);
    }
    if (in) {
      if (p.s != nullptr) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float sj = p.s[c0 + j];
          x[j] = p.divide ? __fmul_rn(x[j], sj) : __fdiv_rn(x[j], sj);
        }
      }
      store32(static_cast<T *>(p.out) + row * p.ldo + c0, p.vec != 0, x);
    }
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
  p.vec = reinterpret_cast<uintptr_t>(a.W) % 16 == 0 && (a.ldw * es) % 16 == 0;
  p.row_groups = row_groups_for((a.M + 127) / 128 * 128, p.units_k);
  const int64_t warps = p.units_k * p.row_groups;
  const dim3 grid((unsigned)((warps + kMxWarps - 1) / kMxWarps));
  const bool fp64 = a.col_scale != nullptr || a.log2b > 0;
  if (a.wt == QAMW_BF16) {
    if (fp64) mx4_quantize_kernel<uint16_t, true><<<grid, 32 * kMxWarps, 0, s>>>(p);
    else mx4_quantize_kernel<uint16_t, false><<<grid, 32 * kMxWarps, 0, s>>>(p);
  } else {
    if (fp64) mx4_quantize_kernel<float, true><<<grid, 32 * kMxWarps, 0, s>>>(p);
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
  p.vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && (a.ldo * es) % 16 == 0;
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
