// Device helpers of the slot kernels: typed element access, slot checks and
// sequence spans.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"

namespace lsq {
namespace dev {

// Elements of an IO-typed array as loaded; converted where they are used, so
// that the next token's are in flight during this one's arithmetic.
template <int IO>
struct Raw {
  using One = uint16_t;
  using Four = uint2;
};
template <>
struct Raw<IO_F32> {
  using One = float;
  using Four = float4;
};

template <int IO>
__device__ __forceinline__ typename Raw<IO>::One raw1(const void* p, int64_t e) {
  return static_cast<const typename Raw<IO>::One*>(p)[e];
}

// Four consecutive elements from e (8-byte aligned; 16 for fp32).
template <int IO>
__device__ __forceinline__ typename Raw<IO>::Four raw4(const void* p, int64_t e) {
  return *reinterpret_cast<const typename Raw<IO>::Four*>(static_cast<const typename Raw<IO>::One*>(p) + e);
}

template <int IO>
__device__ __forceinline__ float widen(typename Raw<IO>::One x) {
  if constexpr (IO == IO_F32) return x;
  else if constexpr (IO == IO_F16) return __half2float(__ushort_as_half(x));
  else return __uint_as_float((uint32_t)x << 16);
}

template <int IO>
__device__ __forceinline__ void widen4(float* dst, typename Raw<IO>::Four x) {
  if constexpr (IO == IO_F32) {
    dst[0] = x.x; dst[1] = x.y; dst[2] = x.z; dst[3] = x.w;
  } else {
    const uint32_t w[2] = {x.x, x.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = widen<IO>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
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
// one beyond the handle or already taken by an earlier entry (the wave's lanes
// compare 64 earlier entries at a time).  works(j) tells whether entry j does
// anything; one that does not takes no slot.  Called by whole waves.
template <typename Works>
__device__ __forceinline__ int slot_of(const int32_t* slots, int i, int n, int lane, Works works) {
  if (!slots) return i < n ? i : kRefused;
  const int s = __builtin_amdgcn_readfirstlane(slots[i]);
  if (s < 0) return kPadded;
  if (s >= n) return kRefused;
  bool taken = false;
  for (int j = lane; j < i; j += 64)
    if (slots[j] == s) taken |= works(j);
  return __any(taken) ? kRefused : s;
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

// The slot of a batch's entry i; an empty sequence takes none.
__device__ __forceinline__ int slot_of(const SlotArgs& a, int i, int lane) {
  return slot_of(a.slots, i, a.nslots, lane, [&](int j) {
    const Span sp = span_of(a, j);
    return sp.t1 > sp.t0;
  });
}

// The destination of a copy's entry i; one whose source is padded or beyond
// its handle takes none.
__device__ __forceinline__ int slot_of(const CopyArgs& a, int i, int lane) {
  return slot_of(a.dst_slots, i, a.dst_n, lane, [&](int j) {
    const int src = a.src_slots ? a.src_slots[j] : j;
    return src >= 0 && src < a.src_n;
  });
}

}  // namespace dev
}  // namespace lsq
