// Slot kernels: the token walk of the recurrence over an fp32 state, and the
// copies between fp32 slots and quantised ones.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"
#include "lsq_slots_dev.h"
#include "lsq_step_impl.h"

namespace lsq {
namespace dev {

// Token walk.  For every token of a sequence, Eq. (1) row by row,
//   S' = fl(S alpha_c),  u = S'.k,  w = fl(beta fl(v - delta u)),
//   S  = fma(w, k_c, S'), o = S.q,
// with the rows in registers from the first token to the last.  Sixteen lanes
// cover a row (lane lc owns columns 4 lc .. 4 lc + 3 of each 64), so that a
// wave's state loads are whole 256-byte runs and both dot products end in a
// 16-lane DPP butterfly; a wave owns 4 R rows, all loaded before the first
// token.  With one token it is the recurrent form: bound by the state's bytes,
// read and written once.
template <int IO, int DK, int DELTA, int DIAG, int R>
__global__ __launch_bounds__(256) void walk_kernel(SlotArgs a, int row_blocks) {
  constexpr int NJ = DK / 64, EPT = DK / 16;
  const int lane = threadIdx.x & 63, lr = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rb = blockIdx.x % row_blocks;
  const int64_t ih = blockIdx.x / row_blocks;
  const int h = (int)(ih % a.heads), i = (int)(ih / a.heads);
  const int row0 = (rb * 4 + wave) * 4 * R;
  if (row0 >= a.dv) return;
  const Span sp = span_of(a, i);
  if (sp.t1 <= sp.t0) return;
  const int slot = slot_of(a.slots, i, a.nslots, lane);
  if (slot == kPadded) return;
  const int orow = row0 + 4 * lc + lr;          // the row whose output this lane stores
  const bool owrite = lc < R && orow < a.dv;
  if (slot == kRefused) {
    if (owrite)
      for (int64_t t = sp.t0; t < sp.t1; ++t)
        store1<IO>(a.o, t * a.o_stride + (int64_t)h * a.dv + orow, __uint_as_float(0x7FC00000u));
    return;
  }
  const bool fresh = a.fresh && a.fresh[i];
  float* S = a.S + ((int64_t)slot * a.heads + h) * a.dv * DK;
  float s[R][EPT];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 4 * r + lr;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!fresh && row < a.dv)
        x = *reinterpret_cast<const float4*>(S + (int64_t)row * DK + 64 * j + 4 * lc);
      s[r][4 * j] = x.x; s[r][4 * j + 1] = x.y; s[r][4 * j + 2] = x.z; s[r][4 * j + 3] = x.w;
    }
  }
  const int64_t hk = (int64_t)(h / a.share) * DK;
  for (int64_t t = sp.t0; t < sp.t1; ++t) {
    float kk[EPT], qq[EPT], aa[DIAG ? EPT : 1], vv[R];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      load4<IO>(&kk[4 * j], a.k, t * a.k_stride + hk + 64 * j + 4 * lc);
      load4<IO>(&qq[4 * j], a.q, t * a.q_stride + hk + 64 * j + 4 * lc);
      if constexpr (DIAG)
        load4<IO_F32>(&aa[4 * j], a.alpha, (t * a.heads + h) * DK + 64 * j + 4 * lc);
    }
    if constexpr (!DIAG) aa[0] = a.alpha[t * a.heads + h];
    const float beta = a.beta[t * a.heads + h];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + 4 * r + lr;
      vv[r] = row < a.dv ? load1<IO>(a.v, t * a.v_stride + (int64_t)h * a.dv + row) : 0.f;
    }
    float out = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float u = 0.f, o = 0.f;
#pragma unroll
      for (int e = 0; e < EPT; ++e) s[r][e] *= aa[DIAG ? e : 0];
      if constexpr (DELTA) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) u = fmaf(s[r][e], kk[e], u);
        u = row_sum<16>(u);
      }
      const float w = beta * (vv[r] - u);
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        s[r][e] = fmaf(w, kk[e], s[r][e]);
        o = fmaf(s[r][e], qq[e], o);
      }
      o = row_sum<16>(o);
      if (lc == r) out = o;
    }
    if (owrite) store1<IO>(a.o, t * a.o_stride + (int64_t)h * a.dv + orow, out);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 4 * r + lr;
    if (row < a.dv) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        *reinterpret_cast<float4*>(S + (int64_t)row * DK + 64 * j + 4 * lc) =
            make_float4(s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]);
    }
  }
}

// Slots -> pages.  A slot's heads are one run of heads*dv*dk elements in both
// handles, so a page is the run's codes and scales, group by group: eight
// consecutive elements per lane, a group's absmax over its group/8 adjacent
// lanes by DPP, the scale, reciprocal and rounding of the calibration.  Bound
// by the fp32 bytes read.
constexpr int kUnits = 4;                        // runs of eight elements per thread

template <int BITS>
__device__ __forceinline__ void quantise8(const float (&x)[8], float inv, uint8_t* codes, int64_t unit) {
  using F = Fmt<BITS>;
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    t[e] = __builtin_amdgcn_fmed3f(fmaf(x[e], inv, F::MQ), F::MQ - F::QMAX, F::MQ + F::QMAX);
  uint32_t X[2];
  pack_block<BITS>(t, X);
  if constexpr (BITS == 4)
    reinterpret_cast<uint32_t*>(codes)[unit] = X[0] ^ F::OFF;
  else
    reinterpret_cast<uint2*>(codes)[unit] = make_uint2(X[0] ^ F::OFF, X[1] ^ F::OFF);
}

template <int BITS>
__global__ __launch_bounds__(256) void store_slots_kernel(CopyArgs a, int64_t units, int blocks) {
  using F = Fmt<BITS>;
  const int i = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int lane = threadIdx.x & 63;
  const int dst = slot_of(a.dst_slots, i, a.dst_n, lane);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  const float* S = a.S + (int64_t)src * units * 8;
  const int gl = a.group / 8;
  float x[kUnits][8];
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    int64_t u = ((int64_t)b * kUnits + n) * 256 + threadIdx.x;
    u = u < units ? u : units - 1;
    load_f32(x[n], S + u * 8);
  }
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = ((int64_t)b * kUnits + n) * 256 + threadIdx.x;
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[n][e]));
    float s = group_max(m, gl) / F::QMAX;
    uint32_t s16 = 0;
    if (a.sfmt != SFMT_F32) {                    // codes are formed with the stored scale
      s16 = scale_to16(s, a.sfmt);
      s = scale_from16(s16, a.sfmt);
    }
    const float inv = inv_scale(s);
    if (u < units) {
      const int64_t to = (int64_t)dst * units + u;
      quantise8<BITS>(x[n], inv, a.codes, to);
      if (u % gl == 0) {
        if (a.sfmt != SFMT_F32)
          static_cast<uint16_t*>(a.scales)[to / gl] = (uint16_t)s16;
        else
          static_cast<float*>(a.scales)[to / gl] = s;
      }
      if (a.ref) store_f32(a.ref + to * 8, x[n]);
    }
  }
}

// One scale per head: a workgroup takes a head, its absmax first, then the
// codes from a second read that the caches serve.
template <int BITS>
__global__ __launch_bounds__(256) void store_head_kernel(CopyArgs a, int head_units) {
  using F = Fmt<BITS>;
  __shared__ float wmax[4];
  const int i = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
  const int dst = slot_of(a.dst_slots, i, a.dst_n, threadIdx.x & 63);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  const float* S = a.S + ((int64_t)src * a.heads + h) * head_units * 8;
  const int64_t to = ((int64_t)dst * a.heads + h) * head_units;
  float x[8], m = 0.f;
  for (int u = threadIdx.x; u < head_units; u += 256) {
    load_f32(x, S + (int64_t)u * 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])) / F::QMAX;
  const float inv = inv_scale(s);
  for (int u = threadIdx.x; u < head_units; u += 256) {
    load_f32(x, S + (int64_t)u * 8);
    quantise8<BITS>(x, inv, a.codes, to + u);
  }
  if (threadIdx.x == 0) static_cast<float*>(a.scales)[(int64_t)dst * a.heads + h] = s;
}

// Pages -> slots: S = fl(C s), eight consecutive elements per lane.  Bound by
// the fp32 bytes written.
template <int BITS>
__global__ __launch_bounds__(256) void load_slots_kernel(CopyArgs a, int64_t units, int blocks,
                                                         int64_t group_units) {
  const int i = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int lane = threadIdx.x & 63;
  const int dst = slot_of(a.dst_slots, i, a.dst_n, lane);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  float* S = a.S + (int64_t)dst * units * 8;
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = ((int64_t)b * kUnits + n) * 256 + threadIdx.x;
    if (u >= units) break;
    const int64_t from = (int64_t)src * units + u;
    const int64_t si = from / group_units;
    const float s = a.sfmt == SFMT_F32
                        ? static_cast<const float*>(a.scales)[si]
                        : scale_from16(static_cast<const uint16_t*>(a.scales)[si], a.sfmt);
    float x[8];
    if constexpr (BITS == 4) {
      const int w = (int)reinterpret_cast<const uint32_t*>(a.codes)[from];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (float)((w << (28 - 4 * e)) >> 28) * s;
    } else {
      const uint2 w = reinterpret_cast<const uint2*>(a.codes)[from];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = (float)(int)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s;
    }
    store_f32(S + u * 8, x);
  }
}

}  // namespace dev

hipError_t launch_walk(const SlotArgs& a, int io, int dk, int delta, int diag, hipStream_t s) {
  constexpr int R = 4;
  const int row_blocks = (a.dv + 16 * R - 1) / (16 * R);
  const int64_t blocks = (int64_t)a.seqs * a.heads * row_blocks;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
#define LSQ_WALK(IO, DK, D, G)                                                                 \
  if (io == IO && dk == DK && delta == D && diag == G) {                                       \
    hipLaunchKernelGGL((dev::walk_kernel<IO, DK, D, G, R>), dim3((unsigned)blocks), dim3(256), \
                       0, s, a, row_blocks);                                                   \
    return hipGetLastError();                                                                  \
  }
#define LSQ_WALK_IO(IO)                                                                  \
  LSQ_WALK(IO, 128, 0, 0) LSQ_WALK(IO, 128, 0, 1) LSQ_WALK(IO, 128, 1, 0)                \
  LSQ_WALK(IO, 128, 1, 1) LSQ_WALK(IO, 64, 0, 0) LSQ_WALK(IO, 64, 0, 1)                  \
  LSQ_WALK(IO, 64, 1, 0) LSQ_WALK(IO, 64, 1, 1)
  LSQ_WALK_IO(IO_F32) LSQ_WALK_IO(IO_F16) LSQ_WALK_IO(IO_BF16)
#undef LSQ_WALK_IO
#undef LSQ_WALK
  return hipErrorInvalidValue;
}

hipError_t launch_store_slots(const CopyArgs& a, int bits, int dk, hipStream_t s) {
  if (a.group == 0) {
    const int64_t blocks = (int64_t)a.count * a.heads;
    if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(256);
    if (bits == 4)
      hipLaunchKernelGGL(dev::store_head_kernel<4>, grid, block, 0, s, a, a.dv * dk / 8);
    else
      hipLaunchKernelGGL(dev::store_head_kernel<8>, grid, block, 0, s, a, a.dv * dk / 8);
    return hipGetLastError();
  }
  const int64_t units = (int64_t)a.heads * a.dv * dk / 8;
  const int64_t per = (units + 256 * dev::kUnits - 1) / (256 * dev::kUnits);
  if (per * a.count > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(per * a.count)), block(256);
  if (bits == 4)
    hipLaunchKernelGGL(dev::store_slots_kernel<4>, grid, block, 0, s, a, units, (int)per);
  else
    hipLaunchKernelGGL(dev::store_slots_kernel<8>, grid, block, 0, s, a, units, (int)per);
  return hipGetLastError();
}

hipError_t launch_load_slots(const CopyArgs& a, int bits, int dk, hipStream_t s) {
  const int64_t units = (int64_t)a.heads * a.dv * dk / 8;
  const int64_t per = (units + 256 * dev::kUnits - 1) / (256 * dev::kUnits);
  const int64_t group_units = a.group ? a.group / 8 : (int64_t)a.dv * dk / 8;
  if (per * a.count > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(per * a.count)), block(256);
  if (bits == 4)
    hipLaunchKernelGGL(dev::load_slots_kernel<4>, grid, block, 0, s, a, units, (int)per, group_units);
  else
    hipLaunchKernelGGL(dev::load_slots_kernel<8>, grid, block, 0, s, a, units, (int)per, group_units);
  return hipGetLastError();
}

}  // namespace lsq
