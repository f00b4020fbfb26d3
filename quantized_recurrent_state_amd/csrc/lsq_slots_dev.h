// Device helpers of the slot kernels: typed element access, slot checks and
// sequence spans.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"

namespace lsq {
namespace dev {

// Element e of an IO-typed array as fp32.
template <int IO>
__device__ __forceinline__ float load1(const void* p, int64_t e) {
  if constexpr (IO == IO_F32) return static_cast<const float*>(p)[e];
  const uint16_t b = static_cast<const uint16_t*>(p)[e];
  if constexpr (IO == IO_F16) return __half2float(__ushort_as_half(b));
  return __uint_as_float((uint32_t)b << 16);
}

// Four consecutive elements from e (8-byte aligned; 16 for fp32).
template <int IO>
__device__ __forceinline__ void load4(float* dst, const void* p, int64_t e) {
  if constexpr (IO == IO_F32) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    dst[0] = x.x; dst[1] = x.y; dst[2] = x.z; dst[3] = x.w;
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + e);
    const uint32_t w[2] = {x.x, x.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
      dst[i] = IO == IO_F16 ? __half2float(__ushort_as_half((unsigned short)b))
                            : __uint_as_float(b << 16);
    }
  }
}

// x rounded once (to nearest, ties to even) to the IO type.
template <int IO>
__device__ __forceinline__ uint16_t to16(float x) {
  static_assert(IO == IO_F16 || IO == IO_BF16, "16-bit types");
  if constexpr (IO == IO_F16) return __half_as_ushort(__float2half_rn(x));
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

template <int IO>
__device__ __forceinline__ void store1(void* p, int64_t e, float x) {
  if constexpr (IO == IO_F32)
    static_cast<float*>(p)[e] = x;
  else
    static_cast<uint16_t*>(p)[e] = to16<IO>(x);
}

constexpr int kPadded = -1, kRefused = -2;

// Entry i's slot: the slot itself, kPadded for a negative one, kRefused for
// one beyond the handle or already named by an earlier entry (the wave's lanes
// compare 64 earlier entries at a time).  Called by whole waves.
__device__ __forceinline__ int slot_of(const int32_t* slots, int i, int n, int lane) {
  if (!slots) return i < n ? i : kRefused;
  const int s = __builtin_amdgcn_readfirstlane(slots[i]);
  if (s < 0) return kPadded;
  if (s >= n) return kRefused;
  bool seen = false;
  for (int j = lane; j < i; j += 64) seen |= slots[j] == s;
  return __any(seen) ? kRefused : s;
}

struct Span {
  int64_t t0, t1;
};

// Entry i's tokens, clamped to the rows there are.
__device__ __forceinline__ Span span_of(const SlotArgs& a, int i) {
  if (!a.cu) return {i, i + 1};
  const int64_t t0 = a.cu[i], t1 = a.cu[i + 1];
  return {t0 < 0 ? 0 : t0 > a.tokens ? a.tokens : t0, t1 < 0 ? 0 : t1 > a.tokens ? a.tokens : t1};
}

}  // namespace dev
}  // namespace lsq
