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
// token, and reads the vectors of D tokens ahead during the current one's sums.
// With one token it is the recurrent form: bound by the state's bytes, read and
// written once (512 slots of 32 heads 128x128 in fp32 with a diagonal decay: 364
// us, 6.0 TB/s; 64 slots in bf16 with the delta rule, some of them fresh: 40 us,
// 5.4 TB/s).  R = 1, 2 and 8 were slower for single tokens.
template <int IO, int DK, int DELTA, int DIAG, int R, int D, bool NT>
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
  const int slot = slot_of(a, i, lane);
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
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      if (!fresh && row < a.dv) x = load_state<NT>(S + (int64_t)row * DK + 64 * j + 4 * lc);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][4 * j + e] = x[e];
    }
  }
  const int64_t hk = (int64_t)(h / a.share) * DK;
  struct Token {
    typename Raw<IO>::Four k[NJ], q[NJ];
    float4 a[DIAG ? NJ : 1];
    typename Raw<IO>::One v[R];
    float alpha, beta;
  };
  auto read = [&](int64_t t) {
    Token x;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      x.k[j] = raw4<IO>(a.k, t * a.k_stride + hk + 64 * j + 4 * lc);
      x.q[j] = raw4<IO>(a.q, t * a.q_stride + hk + 64 * j + 4 * lc);
      if constexpr (DIAG) x.a[j] = raw4<IO_F32>(a.alpha, (t * a.heads + h) * DK + 64 * j + 4 * lc);
    }
    if constexpr (!DIAG) x.alpha = a.alpha[t * a.heads + h];
    x.beta = a.beta[t * a.heads + h];
#pragma unroll
    for (int r = 0; r < R; ++r) {                // rows behind dv repeat the last
      const int row = row0 + 4 * r + lr;
      x.v[r] = raw1<IO>(a.v, t * a.v_stride + (int64_t)h * a.dv + (row < a.dv ? row : a.dv - 1));
    }
    return x;
  };
  Token ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) ring[d] = read(D == 1 || sp.t0 + d < sp.t1 ? sp.t0 + d : sp.t1 - 1);
  auto step = [&](int64_t t, Token& slot) __attribute__((always_inline)) {
    const Token x = slot;
    // no branch around the loads where several tokens are under way: with one the
    // compiler cannot count them and waits for all
    if (D > 1) slot = read(t + D < sp.t1 ? t + D : sp.t1 - 1);
    else if (t + 1 < sp.t1) slot = read(t + 1);
    float kk[EPT], qq[EPT], aa[DIAG ? EPT : 1], vv[R];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      widen4<IO>(&kk[4 * j], x.k[j]);
      widen4<IO>(&qq[4 * j], x.q[j]);
      if constexpr (DIAG) widen4<IO_F32>(&aa[4 * j], x.a[j]);
    }
    if constexpr (!DIAG) aa[0] = x.alpha;
    const float beta = x.beta;
#pragma unroll
    for (int r = 0; r < R; ++r) vv[r] = widen<IO>(x.v[r]);
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
  };
  for (int64_t t = sp.t0; t < sp.t1; t += D) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (t + d < sp.t1) step(t + d, ring[d]);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 4 * r + lr;
    if (row < a.dv) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        store_state<NT>(S + (int64_t)row * DK + 64 * j + 4 * lc,
                        f32x4{s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]});
    }
  }
}

// Slots -> pages.  A slot's heads are one run of heads*dv*dk elements in both
// handles, so a page is the run's codes and scales, group by group: four
// consecutive elements per lane and unit (a wave reads whole 1 KiB runs), a
// group's absmax over its group/4 adjacent lanes, the scale, reciprocal and
// rounding of the calibration.  Bound by the fp32 bytes read (128 slots of 32
// heads 128x128 to INT4 in groups of 32: 59 us, 5.3 TB/s).
constexpr int kUnits = 4;                        // units per thread, all read before the first is used

// Max over an aligned group of gl = 4, 8, 16 or 32 adjacent lanes.
__device__ __forceinline__ float group_max32(float x, int gl) {
  x = group_max(x, gl);
  return gl > 16 ? fmaxf(x, __shfl_xor(x, 16)) : x;
}

template <int BITS>
__device__ __forceinline__ void quantise4(f32x4 x, float inv, uint8_t* codes, int64_t unit) {
  using F = Fmt<BITS>;
  uint32_t t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    t[e] = fbits(__builtin_amdgcn_fmed3f(fmaf(x[e], inv, F::MQ), F::MQ - F::QMAX, F::MQ + F::QMAX));
  if constexpr (BITS == 4)
    reinterpret_cast<uint16_t*>(codes)[unit] =
        (uint16_t)(((t[0] & 0xF) | (t[1] & 0xF) << 4 | (t[2] & 0xF) << 8 | (t[3] & 0xF) << 12) ^ 0x8888u);
  else
    reinterpret_cast<uint32_t*>(codes)[unit] = gather_low_bytes(t[0], t[1], t[2], t[3]) ^ F::OFF;
}

template <int BITS>
__global__ __launch_bounds__(256) void store_slots_kernel(CopyArgs a, int64_t units, int blocks) {
  using F = Fmt<BITS>;
  const int i = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int lane = threadIdx.x & 63;
  const int dst = slot_of(a, i, lane);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  const f32x4* S = reinterpret_cast<const f32x4*>(a.S) + (int64_t)src * units;
  const int gl = a.group / 4;
  const int64_t u0 = (int64_t)b * kUnits * 256 + threadIdx.x;
  f32x4 x[kUnits];
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = u0 + n * 256;
    x[n] = S[u < units ? u : units - 1];
  }
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = u0 + n * 256;
    const float m = fmaxf(fmaxf(fabsf(x[n][0]), fabsf(x[n][1])), fmaxf(fabsf(x[n][2]), fabsf(x[n][3])));
    float s = group_max32(m, gl) / F::QMAX;
    uint32_t s16 = 0;
    if (a.sfmt != SFMT_F32) {                    // codes are formed with the stored scale
      s16 = scale_to16(s, a.sfmt);
      s = scale_from16(s16, a.sfmt);
    }
    const float inv = inv_scale(s);
    if (u < units) {
      const int64_t to = (int64_t)dst * units + u;
      quantise4<BITS>(x[n], inv, a.codes, to);
      if (u % gl == 0) {
        if (a.sfmt != SFMT_F32)
          static_cast<uint16_t*>(a.scales)[to / gl] = (uint16_t)s16;
        else
          static_cast<float*>(a.scales)[to / gl] = s;
      }
      if (a.ref) reinterpret_cast<f32x4*>(a.ref)[to] = x[n];
    }
  }
}

// One scale per head: a workgroup takes a head, its absmax first, then the
// codes from a second read.  Counted, the state is fetched twice: the heads of a
// round do not stay in L2, and the second read comes from the Infinity Cache (128
// slots of 32 heads 128x128: 81 us to INT4, 3.8 TB/s of the bytes counted once, and
// 90 to INT8; one slot 9.7 us).
template <int BITS>
__global__ __launch_bounds__(256) void store_head_kernel(CopyArgs a, int head_units) {
  using F = Fmt<BITS>;
  __shared__ float wmax[4];
  const int i = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
  const int dst = slot_of(a, i, threadIdx.x & 63);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  const f32x4* S = reinterpret_cast<const f32x4*>(a.S) + ((int64_t)src * a.heads + h) * head_units;
  const int64_t to = ((int64_t)dst * a.heads + h) * head_units;
  float m = 0.f;
  for (int u = threadIdx.x; u < head_units; u += 256) {
    const f32x4 x = S[u];
    m = fmaxf(m, fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
  __syncthreads();
  const float s = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3])) / F::QMAX;
  const float inv = inv_scale(s);
  for (int u = threadIdx.x; u < head_units; u += 256) quantise4<BITS>(S[u], inv, a.codes, to + u);
  if (threadIdx.x == 0) static_cast<float*>(a.scales)[(int64_t)dst * a.heads + h] = s;
}

// Pages -> slots: S = fl(C s), four consecutive elements per lane and unit.
// Bound by the fp32 bytes written (128 slots as above: 48 us, 6.5 TB/s with
// the codes in the last-level cache; 256 slots of INT8 from memory: 125 us, 5.4).
template <int BITS, bool NT>
__global__ __launch_bounds__(256) void load_slots_kernel(CopyArgs a, int64_t units, int blocks,
                                                         int64_t group_units) {
  const int i = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int lane = threadIdx.x & 63;
  const int dst = slot_of(a, i, lane);
  const int src = a.src_slots ? a.src_slots[i] : i;
  if (dst < 0 || src < 0 || src >= a.src_n) return;
  f32x4* S = reinterpret_cast<f32x4*>(a.S) + (int64_t)dst * units;
  const int64_t u0 = (int64_t)b * kUnits * 256 + threadIdx.x;
  uint32_t w[kUnits];
  float s[kUnits];
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = u0 + n * 256;
    const int64_t from = (int64_t)src * units + (u < units ? u : units - 1), si = from / group_units;
    w[n] = BITS == 4 ? reinterpret_cast<const uint16_t*>(a.codes)[from]
                     : reinterpret_cast<const uint32_t*>(a.codes)[from];
    s[n] = a.sfmt == SFMT_F32 ? static_cast<const float*>(a.scales)[si]
                              : scale_from16(static_cast<const uint16_t*>(a.scales)[si], a.sfmt);
  }
#pragma unroll
  for (int n = 0; n < kUnits; ++n) {
    const int64_t u = u0 + n * 256;
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[e] = (float)((int)(w[n] << (32 - BITS - BITS * e)) >> (32 - BITS)) * s[n];
    if (u < units) store_state<NT>(reinterpret_cast<float*>(S + u), x);
  }
}

}  // namespace dev

namespace {

template <int IO, int DK, int DELTA, int DIAG>
hipError_t launch_walk_instance(const SlotArgs& a, int nt, hipStream_t s) {
  auto launch = [&](auto kernel, int R) {
    const int row_blocks = (a.dv + 16 * R - 1) / (16 * R);
    const int64_t blocks = (int64_t)a.seqs * a.heads * row_blocks;
    if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, row_blocks);
    return hipGetLastError();
  };
  if (!a.cu)
    return nt ? launch(dev::walk_kernel<IO, DK, DELTA, DIAG, 4, 1, true>, 4)
              : launch(dev::walk_kernel<IO, DK, DELTA, DIAG, 4, 1, false>, 4);
  // Prompts: a token's chain of sums is what takes the time, so rows are spread
  // over waves while the workgroups do not share CUs (one prompt of 32 heads
  // 128x128 in bf16 with the delta rule: 0.43 us per token with R = 2, 0.56 with
  // 4; 16 prompts: 1.53 and 1.44), and two tokens are read ahead (0.56 and, with
  // one, 0.60; of a diagonal decay 0.52 and 0.60).
  const bool few = (int64_t)a.seqs * a.heads * ((a.dv + 31) / 32) <= 256;
  return few ? launch(dev::walk_kernel<IO, DK, DELTA, DIAG, 2, 2, false>, 2)
             : launch(dev::walk_kernel<IO, DK, DELTA, DIAG, 4, 2, false>, 4);
}

template <int IO, int DK>
hipError_t launch_walk_rule(const SlotArgs& a, int delta, int diag, int nt, hipStream_t s) {
  if (delta) return diag ? launch_walk_instance<IO, DK, 1, 1>(a, nt, s) : launch_walk_instance<IO, DK, 1, 0>(a, nt, s);
  return diag ? launch_walk_instance<IO, DK, 0, 1>(a, nt, s) : launch_walk_instance<IO, DK, 0, 0>(a, nt, s);
}

}  // namespace

hipError_t launch_walk(const SlotArgs& a, int io, int dk, int delta, int diag, int nt, hipStream_t s) {
  if (io == IO_F32) return dk == 128 ? launch_walk_rule<IO_F32, 128>(a, delta, diag, nt, s) : launch_walk_rule<IO_F32, 64>(a, delta, diag, nt, s);
  if (io == IO_F16) return dk == 128 ? launch_walk_rule<IO_F16, 128>(a, delta, diag, nt, s) : launch_walk_rule<IO_F16, 64>(a, delta, diag, nt, s);
  return dk == 128 ? launch_walk_rule<IO_BF16, 128>(a, delta, diag, nt, s) : launch_walk_rule<IO_BF16, 64>(a, delta, diag, nt, s);
}

hipError_t launch_store_slots(const CopyArgs& a, int bits, int dk, hipStream_t s) {
  if (a.group == 0) {
    const int64_t blocks = (int64_t)a.count * a.heads;
    if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(256);
    if (bits == 4)
      hipLaunchKernelGGL(dev::store_head_kernel<4>, grid, block, 0, s, a, a.dv * dk / 4);
    else
      hipLaunchKernelGGL(dev::store_head_kernel<8>, grid, block, 0, s, a, a.dv * dk / 4);
    return hipGetLastError();
  }
  const int64_t units = (int64_t)a.heads * a.dv * dk / 4;
  const int64_t per = (units + 256 * dev::kUnits - 1) / (256 * dev::kUnits);
  if (!fits_launch(per * a.count, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(per * a.count)), block(256);
  if (bits == 4)
    hipLaunchKernelGGL(dev::store_slots_kernel<4>, grid, block, 0, s, a, units, (int)per);
  else
    hipLaunchKernelGGL(dev::store_slots_kernel<8>, grid, block, 0, s, a, units, (int)per);
  return hipGetLastError();
}

hipError_t launch_load_slots(const CopyArgs& a, int bits, int dk, hipStream_t s) {
  const int64_t units = (int64_t)a.heads * a.dv * dk / 4;
  const int64_t per = (units + 256 * dev::kUnits - 1) / (256 * dev::kUnits);
  const int64_t group_units = a.group ? a.group / 4 : (int64_t)a.dv * dk / 4;
  if (!fits_launch(per * a.count, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(per * a.count)), block(256);
  const auto kernel = bits == 4 ? (a.nt ? dev::load_slots_kernel<4, true> : dev::load_slots_kernel<4, false>)
                                : (a.nt ? dev::load_slots_kernel<8, true> : dev::load_slots_kernel<8, false>);
  hipLaunchKernelGGL(kernel, grid, block, 0, s, a, units, (int)per, group_units);
  return hipGetLastError();
}

}  // namespace lsq
