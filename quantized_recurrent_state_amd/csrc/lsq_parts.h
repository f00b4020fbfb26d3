// Device helpers of the kernels that run fp32 work on the bf16 matrix cores:
// values as sums of bf16 parts, and the decays' logarithms.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots_dev.h"

namespace lsq {
namespace dev {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// x as a sum of N bf16 parts, four values at a time.  (The differences by the
// bf16 dot product, half as many instructions, take longer: 337 us instead of 326
// for 16 x 2560 tokens of 32 heads 128x128 in bf16.)
template <int N>
__device__ __forceinline__ void split4(f32x4 x, bf16x4 (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x[2 * h], x[2 * h + 1]}, bf16x2));
      if (i + 1 < N) {
        x[2 * h] -= __uint_as_float(w[h] << 16);
        x[2 * h + 1] -= __uint_as_float(w[h] & 0xFFFF0000u);
      }
    }
    p[i] = __builtin_bit_cast(bf16x4, (uint64_t)w[1] << 32 | w[0]);
  }
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Two values rounded once to a 16-bit type.
template <int IO>
__device__ __forceinline__ uint32_t pair16(float x, float y) {
  if constexpr (IO == IO_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
  else return to16<IO_F16>(x) | (uint32_t)to16<IO_F16>(y) << 16;
}

// Four values of a column from four consecutive rows of a row-major LDS tile:
// lane 16 g + i points at row 4 g + i / 4, column 4 (i % 4) of a 16 x 16 block
// and receives rows 4 g .. 4 g + 3 of column i.
__device__ __forceinline__ bf16x4 read_column4(const __bf16* p) {
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                        (__attribute__((address_space(3))) s16x4*)p));
}

// 2^x of a double, to fp32.
__device__ __forceinline__ float exp2_of(double x) {
  const float h = (float)x;
  return __builtin_amdgcn_exp2f(h) * (1.f + 0.69314718f * (float)(x - (double)h));
}

// log2(x) of 0 <= x, to 2^-26 of itself, also next to one; -160 for 0
// and subnormals, NaN for negative x and NaN.  x = 2^e (1 + f) with 1 + f
// from sqrt(1/2) to sqrt(2), log2(1 + f) = 2 / ln 2 atanh(s), s = f / (2 + f) in
// |s| <= 0.1716: atanh(s) = s (1 + s^2/3 + s^4/5 + ...), the bracket's tail in
// fp32 (its rounding is scaled by s^2), s and the product with 2 / ln 2 as sums
// of two floats.  A library log2 in fp64 cost 2 us per round on the critical
// path of a chunk.
__device__ __forceinline__ double log2_of(float x) {
  float m = __builtin_amdgcn_frexp_mantf(x);     // in [1/2, 1)
  int e = __builtin_amdgcn_frexp_expf(x);
  if (m < 0.70710678f) {
    m *= 2.f;
    --e;
  }
  const float f = m - 1.f;                       // exact
  const float t = 2.f + f, tl = (2.f - t) + f;   // t + tl = 2 + f
  const float r = __builtin_amdgcn_rcpf(t);
  const float s = f * r;
  const float sl = (fmaf(-s, t, f) - s * tl) * r;   // s + sl = f / (2 + f)
  const float z = s * s;
  const float tail = z * fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 13, 1.f / 11), 1.f / 9), 1.f / 7), 0.2f), 1.f / 3);
  constexpr float C = 2.8853900817779268f, CL = (float)(2.8853900817779268 - (double)C);   // 2 / ln 2
  const float h = C * s;
  const float l = fmaf(C, s, -h) + (fmaf(CL, s, C * sl) + h * tail);
  double y = (double)e + ((double)h + (double)l);
  if (!(x >= 0x1p-126f)) y = x >= 0.f ? -160.0 : __builtin_nan("");   // 0 and subnormals count as 0
  return y;
}

}  // namespace dev
}  // namespace lsq
