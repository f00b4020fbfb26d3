// Chunked linear attention with a scalar decay per head (delta 0) on the
// matrix cores: packed prompts from and into the slots of an fp32 handle.
//
// Within a chunk of C tokens, with c_t the product of the decays up to t,
//   P[t,s] = (q_t.k_s) c_t / c_s beta_s              (s <= t, else 0)
//   o_t    = c_t S q_t + sum_s P[t,s] v_s
//   S      = c_C S + sum_s (c_C / c_s) beta_s v_s k_s^T.
// The ratios are 2^(L_t - L_s) of sums L of log2(alpha), formed in fp64 and
// held as two floats, so that a difference is exact to fp32 for decays near
// one and for products far below the range of fp32 alike; alpha = 0 counts as
// 2^-160, whose every product with a finite number is 0 in fp32.
//
// Precision.  The bf16 MFMA is the fast one, so every operand is a sum of
// bf16 parts: q, k and v of bf16 inputs are one part, of binary16 two, of fp32
// three (each exact), computed operands (P, S, the scaled v) are split into as
// many as their use needs, and the products of parts i + j < N are added, N = 3
// for the state and for fp32 outputs (relative 2^-24), N = 2 for 16-bit
// outputs (2^-16, against their own half step of 2^-8 or 2^-11).  One rounded
// part instead would cost half a step of bf16 in the state at every chunk.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"
#include "lsq_slots_dev.h"

namespace lsq {
namespace dev {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Tiling of one instance.  NW waves own 16 value columns each.
template <int IO, int DK, int NW>
struct Tile {
  static constexpr int NP = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3;   // parts of an input
  static constexpr int NO = IO == IO_F32 ? 3 : 2;                       // parts on the output's side
  static constexpr int C = IO == IO_BF16 ? 64 : 32;                     // tokens per chunk
  static constexpr int DV = 16 * NW, NT = 64 * NW;
  static constexpr int EU = IO == IO_F32 ? 4 : 8;                       // elements of a 16-byte unit
  // LDS row pitches in elements: rows 32 bytes apart in the banks
  static constexpr int PK = DK + 16, PV = DV + 16, PP = C + 8;
  static constexpr int QU = (C * DK / EU + NT - 1) / NT;                // units of q (of k) per thread
  static constexpr int VU = C * DV / EU / NT;
  static constexpr bool QGUARD = QU * NT > C * DK / EU;
};

// x as a sum of N bf16 parts, four values at a time.
template <int N>
__device__ __forceinline__ void split4(f32x4 x, bf16x4 (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = __builtin_convertvector(x, bf16x4);
    if (i + 1 < N) x = x - __builtin_convertvector(p[i], f32x4);
  }
}

__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Four values of a column from four consecutive rows of a row-major LDS tile:
// lane 16 g + i points at row 4 g + i / 4, column 4 (i % 4) of a 16 x 16 block
// and receives rows 4 g .. 4 g + 3 of column i.
__device__ __forceinline__ bf16x4 read_column4(const __bf16* p) {
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                        (__attribute__((address_space(3))) s16x4*)p));
}

// Decays of one chunk, per token.
template <int C>
struct Decays {
  float hi[C], lo[C];      // L_t, the sum of log2(alpha) from the chunk's start
  float beta[C];
  float cin[C];            // c_t = 2^L_t
  float w[C];              // (c_C / c_t) beta_t
  float gamma;             // c_C
};

// One wave fills them from its lanes' tokens (alpha 1 and beta 0 behind the
// sequence); returns L_C.
template <int C>
__device__ __forceinline__ double fill_decays(Decays<C>& d, float alpha, float beta, int lane) {
  double l = log2((double)alpha);
  l = l < -160.0 ? -160.0 : l;
#pragma unroll
  for (int o = 1; o < C; o *= 2) {
    const double up = __shfl_up(l, o);
    if (lane >= o) l += up;
  }
  const double end = __shfl(l, C - 1);
  if (lane < C) {
    const float hi = (float)l;
    d.hi[lane] = hi;
    d.lo[lane] = (float)(l - (double)hi);
    d.beta[lane] = beta;
    d.cin[lane] = exp2f(hi) * (1.f + 0.69314718f * d.lo[lane]);
    const double r = end - l;
    const float rh = (float)r;
    d.w[lane] = exp2f(rh) * (1.f + 0.69314718f * (float)(r - (double)rh)) * beta;
    if (lane == C - 1) d.gamma = d.cin[lane];
  }
  return end;
}

// The segment a workgroup takes: sequence i, its j-th of n segments.  With a
// segment length L, sequence i's segments begin at number cu[i] / L + i (its
// length over L rounded up is at most the distance to the next).
struct Segment {
  int i, j, n;
  int64_t t0, t1;
};

__device__ __forceinline__ Segment segment_of(const SlotArgs& a, int64_t L, int64_t s) {
  Segment g{};
  if (L == 0) {
    g.i = (int)s;
  } else {
    int lo = 0, hi = a.seqs - 1;             // the last sequence that begins at or before s
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (span_of(a, mid).t0 / L + mid <= s) lo = mid; else hi = mid - 1;
    }
    g.i = lo;
  }
  const Span sp = span_of(a, g.i);
  const int64_t len = sp.t1 > sp.t0 ? sp.t1 - sp.t0 : 0;
  if (L == 0) {
    g.n = len > 0;
    g.t0 = sp.t0;
    g.t1 = sp.t1;
  } else {
    const int64_t j = s - (sp.t0 / L + g.i);
    g.n = (int)((len + L - 1) / L);
    g.j = j < 0 || j >= g.n ? g.n : (int)j;
    g.t0 = sp.t0 + (int64_t)g.j * L;
    g.t1 = g.t0 + L < sp.t1 ? g.t0 + L : sp.t1;
  }
  return g;
}

// Block number -> work item, neighbours in one XCD (blocks go to the eight
// XCDs in turn): heads that share q and k then share an L2.
__device__ __forceinline__ int64_t xcd_item(int64_t b, int64_t n) {
  const int64_t q = n / 8, r = n % 8, x = b % 8, p = b / 8;
  return x * q + (x < r ? x : r) + p;
}

// One workgroup walks the chunks of one segment of one head, 16 NW value
// columns of it.  Per chunk: the chunk's rows (read one chunk ahead into
// registers) go to LDS as bf16 parts; the waves share out P's lower tiles; then
// each wave has its 16 columns of S in registers in the layout that the MFMA
// both writes (S^T[dk, dv] accumulated from k^T and the scaled v) and reads (as
// the operand of S q): the k index of an operand is only a labelling, so slots
// 0-3 and 4-7 of a lane group g stand for rows 4 g .. and 16 + 4 g .. of a
// 32-row step in every product.  OUT = false adds up a segment's writes alone
// (no q, no output), for the segments behind it.
template <int IO, int DK, int NW, bool OUT>
__global__ __launch_bounds__(64 * NW) void attend_kernel(AttendArgs args) {
  using T = Tile<IO, DK, NW>;
  constexpr int NP = T::NP, NO = T::NO, C = T::C, PK = T::PK, PV = T::PV, PP = T::PP;
  constexpr int CT = C / 16, KT = DK / 16, KB = C / 32;
  const SlotArgs& a = args.s;
  __shared__ __align__(16) __bf16 kl[NP][C * PK];
  __shared__ __align__(16) __bf16 vl[NP][C * PV];
  __shared__ __align__(16) __bf16 ql[OUT ? NP : 1][OUT ? C * PK : 8];
  __shared__ __align__(16) __bf16 pl[OUT ? NO : 1][OUT ? C * PP : 8];
  __shared__ __align__(16) Decays<C> dec[2];

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t item = xcd_item(blockIdx.x, gridDim.x);
  const int slice = (int)(item % args.slices);
  const int h = (int)(item / args.slices % a.heads);
  const int64_t seg = item / args.slices / a.heads;
  const Segment sg = segment_of(a, args.seg_len, seg);
  if (sg.j >= sg.n || (!OUT && sg.j == sg.n - 1)) return;
  const int slot = slot_of(a.slots, sg.i, a.nslots, lane);
  if (slot == kPadded) return;
  const int d0 = slice * T::DV + 16 * wave;      // the wave's first value column
  if (slot == kRefused) {
    if (OUT)
      for (int64_t t = sg.t0; t < sg.t1; ++t)
        for (int c = tid; c < T::DV; c += T::NT)
          if (slice * T::DV + c < a.dv)
            store1<IO>(a.o, t * a.o_stride + (int64_t)h * a.dv + slice * T::DV + c,
                       __uint_as_float(0x7FC00000u));
    return;
  }

  // ---- the chunk's rows, 16 bytes per unit
  const int64_t hk = (int64_t)(h / a.share) * DK, hv = (int64_t)h * a.dv + slice * T::DV;
  const int vcols = a.dv - slice * T::DV < T::DV ? a.dv - slice * T::DV : T::DV;
  uint4 rq[OUT ? T::QU : 1], rk[T::QU], rv[T::VU];
  float ra = 1.f, rb = 0.f;
  auto read_chunk = [&](int64_t t0) {
    const int live = (int)(sg.t1 - t0 < C ? sg.t1 - t0 : C);
    if (wave == NW - 1) {
      ra = lane < live ? a.alpha[(t0 + lane) * a.heads + h] : 1.f;
      rb = lane < live ? a.beta[(t0 + lane) * a.heads + h] : 0.f;
    }
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n = 0; n < T::QU; ++n) {
      const int u = n * T::NT + tid, row = u / (DK / T::EU), col = u % (DK / T::EU) * T::EU;
      const bool in = row < live;
      constexpr int B = 16 / T::EU;
      rk[n] = in ? *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) +
                                                   ((t0 + row) * a.k_stride + hk + col) * B) : zero;
      if constexpr (OUT)
        rq[n] = in ? *reinterpret_cast<const uint4*>(static_cast<const char*>(a.q) +
                                                     ((t0 + row) * a.q_stride + hk + col) * B) : zero;
    }
#pragma unroll
    for (int n = 0; n < T::VU; ++n) {
      const int u = n * T::NT + tid, row = u / (T::DV / T::EU), col = u % (T::DV / T::EU) * T::EU;
      constexpr int B = 16 / T::EU;
      const int64_t e = (t0 + row) * a.v_stride + hv + col;
      rv[n] = zero;
      if (row < live) {
        if (args.v_wide) {
          if (col < vcols) rv[n] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + e * B);
        } else {                                 // odd widths or addresses: by element
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int x = 0; x < T::EU; ++x)
            if (col + x < vcols) {
              if constexpr (IO == IO_F32)
                w[x] = static_cast<const uint32_t*>(a.v)[e + x];
              else
                w[x / 2] |= (uint32_t)static_cast<const uint16_t*>(a.v)[e + x] << (16 * (x & 1));
            }
          rv[n] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  };
  auto put = [&](uint4 r, auto* dst, int row, int pitch, int col) {   // one unit's parts
    __bf16* p = &dst[0][row * pitch + col];
    constexpr int plane = sizeof(dst[0]) / sizeof(__bf16);
    if constexpr (IO == IO_BF16) {
      *reinterpret_cast<uint4*>(p) = r;
    } else if constexpr (IO == IO_F32) {
      bf16x4 s[NP];
      split4<NP>(__builtin_bit_cast(f32x4, r), s);
#pragma unroll
      for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x4*>(p + i * plane) = s[i];
    } else {
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = __half2float(__ushort_as_half((unsigned short)(w[2 * q + e / 2] >> (16 * (e & 1)))));
        bf16x4 s[NP];
        split4<NP>(x, s);
#pragma unroll
        for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x4*>(p + i * plane + 4 * q) = s[i];
      }
    }
  };

  // ---- the state's columns: lane li has column d0 + li, rows 16 I + 4 g + v of S^T
  f32x4 S[KT];
  const bool own = 16 * wave + li < vcols;
  const int64_t state = ((int64_t)h * a.dv + d0 + li) * DK + 4 * g, per = (int64_t)a.heads * a.dv * DK;
  float* slot_S = a.S + slot * per + state;
  float* seg_S = args.ws + seg * per + state;
  {
    const bool from_ws = OUT && sg.n > 1;
    const bool zero = !OUT || (!from_ws && a.fresh && a.fresh[sg.i]);
    const float* p = from_ws ? seg_S : slot_S;
#pragma unroll
    for (int I = 0; I < KT; ++I)
      S[I] = own && !zero ? *reinterpret_cast<const f32x4*>(p + 16 * I) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if constexpr (OUT)                             // the tiles above the diagonal stay zero
    for (int e = tid; e < NO * C * PP / 2; e += T::NT) reinterpret_cast<uint32_t*>(&pl[0][0])[e] = 0;

  double total = 0.0;
  read_chunk(sg.t0);
  if (wave == NW - 1) total += fill_decays<C>(dec[0], ra, rb, lane);
  int buf = 0;
  for (int64_t t0 = sg.t0; t0 < sg.t1; t0 += C, buf ^= 1) {
    const bool more = t0 + C < sg.t1;
#pragma unroll
    for (int n = 0; n < T::QU; ++n) {
      const int u = n * T::NT + tid, row = u / (DK / T::EU), col = u % (DK / T::EU) * T::EU;
      if (!T::QGUARD || row < C) {
        put(rk[n], kl, row, PK, col);
        if constexpr (OUT) put(rq[n], ql, row, PK, col);
      }
    }
#pragma unroll
    for (int n = 0; n < T::VU; ++n) {
      const int u = n * T::NT + tid, row = u / (T::DV / T::EU), col = u % (T::DV / T::EU) * T::EU;
      put(rv[n], vl, row, PV, col);
    }
    __syncthreads();
    if (more) read_chunk(t0 + C);
    const Decays<C>& d = dec[buf];
    if constexpr (OUT) {
      // ---- P^T tiles: rows s, columns t
      for (int idx = wave; idx < CT * (CT + 1) / 2; idx += NW) {
        const int ti = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0, si = idx - ti * (ti + 1) / 2;
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) {
          bf16x8 kp[NP], qp[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            kp[i] = *reinterpret_cast<const bf16x8*>(&kl[i][(16 * si + li) * PK + 32 * ks + 8 * g]);
            qp[i] = *reinterpret_cast<const bf16x8*>(&ql[i][(16 * ti + li) * PK + 32 * ks + 8 * g]);
          }
#pragma unroll
          for (int i = NP - 1; i >= 0; --i)      // small products first
#pragma unroll
            for (int j = NP - 1; j >= 0; --j)
              if (i + j < NO) acc = mfma(kp[i], qp[j], acc);
        }
        const int t = 16 * ti + li, s0 = 16 * si + 4 * g;
        const float ht = d.hi[t], lt = d.lo[t];
        const f32x4 hs = *reinterpret_cast<const f32x4*>(&d.hi[s0]), ls = *reinterpret_cast<const f32x4*>(&d.lo[s0]);
        const f32x4 bs = *reinterpret_cast<const f32x4*>(&d.beta[s0]);
        f32x4 p;
#pragma unroll
        for (int v = 0; v < 4; ++v)
          p[v] = s0 + v <= t ? acc[v] * (__builtin_amdgcn_exp2f((ht - hs[v]) + (lt - ls[v])) * bs[v]) : 0.f;
        bf16x4 parts[NO];
        split4<NO>(p, parts);
#pragma unroll
        for (int i = 0; i < NO; ++i) *reinterpret_cast<bf16x4*>(&pl[i][t * PP + s0]) = parts[i];
      }
      __syncthreads();
    }
    // ---- the wave's 16 columns of v, by columns
    bf16x4 vr[KB][2][NP];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int i = 0; i < NP; ++i)
          vr[kb][y][i] = read_column4(&vl[i][(32 * kb + 16 * y + 4 * g + li / 4) * PV + 16 * wave + 4 * (li % 4)]);
    if constexpr (OUT) {
      // ---- o^T tiles: rows dv, columns t
      f32x4 acc[CT];
#pragma unroll
      for (int ti = 0; ti < CT; ++ti) acc[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < DK / 32; ++ks) {
        bf16x4 s0[NO], s1[NO];
        split4<NO>(S[2 * ks], s0);
        split4<NO>(S[2 * ks + 1], s1);
#pragma unroll
        for (int ti = 0; ti < CT; ++ti) {
          bf16x8 qp[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const __bf16* p = &ql[i][(16 * ti + li) * PK + 32 * ks + 4 * g];
            qp[i] = join(*reinterpret_cast<const bf16x4*>(p), *reinterpret_cast<const bf16x4*>(p + 16));
          }
#pragma unroll
          for (int i = NO - 1; i >= 0; --i)
#pragma unroll
            for (int j = NP - 1; j >= 0; --j)
              if (i + j < NO) acc[ti] = mfma(join(s0[i], s1[i]), qp[j], acc[ti]);
        }
      }
#pragma unroll
      for (int ti = 0; ti < CT; ++ti) {
        const float c = d.cin[16 * ti + li];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[ti][v] *= c;
#pragma unroll
        for (int kb = 0; kb <= ti / 2; ++kb) {
          bf16x8 pp[NO];
#pragma unroll
          for (int i = 0; i < NO; ++i) {
            const __bf16* p = &pl[i][(16 * ti + li) * PP + 32 * kb + 4 * g];
            pp[i] = join(*reinterpret_cast<const bf16x4*>(p), *reinterpret_cast<const bf16x4*>(p + 16));
          }
#pragma unroll
          for (int i = NO - 1; i >= 0; --i)
#pragma unroll
            for (int j = NP - 1; j >= 0; --j)
              if (i + j < NO) acc[ti] = mfma(join(vr[kb][0][j], vr[kb][1][j]), pp[i], acc[ti]);
        }
        const int64_t t = t0 + 16 * ti + li;
        const int c0 = 16 * wave + 4 * g;
        if (t < sg.t1) {
          const int64_t e = t * a.o_stride + hv + c0;
          if (args.o_wide) {
            if (c0 < vcols) {
              if constexpr (IO == IO_F32) {
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.o) + e) = acc[ti];
              } else {
                const uint32_t w0 = to16<IO>(acc[ti][0]) | (uint32_t)to16<IO>(acc[ti][1]) << 16;
                const uint32_t w1 = to16<IO>(acc[ti][2]) | (uint32_t)to16<IO>(acc[ti][3]) << 16;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + e) = make_uint2(w0, w1);
              }
            }
          } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (c0 + v < vcols) store1<IO>(a.o, e + v, acc[ti][v]);
          }
        }
      }
    }
    // ---- S = c_C S + k^T (w v)
    bf16x8 vs[KB][3];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      bf16x4 half[2][3];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        f32x4 x = __builtin_convertvector(vr[kb][y][0], f32x4);
#pragma unroll
        for (int i = 1; i < NP; ++i) x = x + __builtin_convertvector(vr[kb][y][i], f32x4);
        x = x * *reinterpret_cast<const f32x4*>(&d.w[32 * kb + 16 * y + 4 * g]);
        split4<3>(x, half[y]);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) vs[kb][i] = join(half[0][i], half[1][i]);
    }
    const float gamma = d.gamma;
#pragma unroll
    for (int I = 0; I < KT; ++I) {
      S[I] = S[I] * gamma;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        bf16x8 kp[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const __bf16* p = &kl[i][(32 * kb + 4 * g + li / 4) * PK + 16 * I + 4 * (li % 4)];
          kp[i] = join(read_column4(p), read_column4(p + 16 * PK));
        }
#pragma unroll
        for (int i = NP - 1; i >= 0; --i)
#pragma unroll
          for (int j = 2; j >= 0; --j)
            if (i + j < 3) S[I] = mfma(kp[i], vs[kb][j], S[I]);
      }
    }
    if (more && wave == NW - 1) total += fill_decays<C>(dec[buf ^ 1], ra, rb, lane);
    __syncthreads();
  }

  if (own && (!OUT || sg.j == sg.n - 1)) {
    float* p = OUT ? slot_S : seg_S;
#pragma unroll
    for (int I = 0; I < KT; ++I) *reinterpret_cast<f32x4*>(p + 16 * I) = S[I];
  }
  if (!OUT && slice == 0 && tid == 64 * (NW - 1)) args.ws_decay[seg * a.heads + h] = exp2f((float)total);
}

// The states before each segment of a sequence of several: S_0 is the slot's
// (or 0), S_{j+1} = decay_j S_j + writes_j; segment j's writes are replaced by
// S_j.  One thread per four elements of a head, one pass over the segments.
__global__ __launch_bounds__(256) void combine_kernel(AttendArgs args, int blocks, int64_t quads) {
  const SlotArgs& a = args.s;
  const int lane = threadIdx.x & 63;
  const int b = blockIdx.x % blocks, i = blockIdx.x / blocks;
  const Span sp = span_of(a, i);
  const int64_t L = args.seg_len, first = sp.t0 / L + i;
  const int64_t n = sp.t1 > sp.t0 ? (sp.t1 - sp.t0 + L - 1) / L : 0;
  if (n < 2) return;
  const int slot = slot_of(a.slots, i, a.nslots, lane);
  const int64_t q = (int64_t)b * 256 + threadIdx.x;     // quad of the sequence's states
  if (slot < 0 || q >= quads) return;
  const int h = (int)(q / (quads / a.heads));
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (!(a.fresh && a.fresh[i])) S = reinterpret_cast<const f32x4*>(a.S)[slot * quads + q];
  f32x4* ws = reinterpret_cast<f32x4*>(args.ws) + first * quads + q;
  f32x4 x = ws[0];
  for (int64_t j = 0; j < n; ++j) {
    ws[j * quads] = S;
    if (j + 1 < n) {
      const f32x4 next = j + 2 < n ? ws[(j + 1) * quads] : x;   // the last segment's writes are not needed
      S = S * args.ws_decay[(first + j) * a.heads + h] + x;
      x = next;
    }
  }
}

}  // namespace dev

namespace {

template <int IO, int DK, int NW>
hipError_t launch_instance(const AttendArgs& args, unsigned blocks, hipStream_t s) {
  const SlotArgs& a = args.s;
  if (args.seg_len) {
    hipLaunchKernelGGL((dev::attend_kernel<IO, DK, NW, false>), dim3(blocks), dim3(64 * NW), 0, s, args);
    const int64_t quads = (int64_t)a.heads * a.dv * DK / 4, per = (quads + 255) / 256;
    if (per * a.seqs > INT32_MAX) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(dev::combine_kernel, dim3((unsigned)(per * a.seqs)), dim3(256), 0, s, args,
                       (int)per, quads);
  }
  hipLaunchKernelGGL((dev::attend_kernel<IO, DK, NW, true>), dim3(blocks), dim3(64 * NW), 0, s, args);
  return hipGetLastError();
}

template <int IO, int DK>
hipError_t launch_width(const AttendArgs& args, unsigned blocks, hipStream_t s) {
  return args.s.dv <= 64 ? launch_instance<IO, DK, 4>(args, blocks, s)
                         : launch_instance<IO, DK, 8>(args, blocks, s);
}

}  // namespace

#ifndef LSQ_ATT_TARGET
#define LSQ_ATT_TARGET 1024
#endif
#ifndef LSQ_ATT_MIN
#define LSQ_ATT_MIN 512
#endif

AttendPlan attend_plan(int64_t tokens, int32_t seqs, int32_t heads, int32_t dk, int32_t dv) {
  AttendPlan p{};
  p.slices = (dv + 127) / 128;
  const int64_t rows = (int64_t)heads * p.slices;
  int64_t L = (tokens * rows / LSQ_ATT_TARGET + 63) / 64 * 64;
  if (L < LSQ_ATT_MIN) L = LSQ_ATT_MIN;
  p.segments = seqs;
  if (L < tokens) {
    p.seg_len = L;
    p.segments = tokens / L + seqs;
    const int64_t state = (int64_t)heads * dv * dk * 4;
    p.state_bytes = p.segments * state;
    p.workspace = (size_t)(p.state_bytes + p.segments * heads * 4);
  }
  return p;
}

hipError_t launch_attend(const AttendArgs& args, int64_t segments, int io, int dk, hipStream_t s) {
  const int64_t blocks = segments * args.s.heads * args.slices;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  const unsigned n = (unsigned)blocks;
  if (io == IO_F32) return dk == 128 ? launch_width<IO_F32, 128>(args, n, s) : launch_width<IO_F32, 64>(args, n, s);
  if (io == IO_F16) return dk == 128 ? launch_width<IO_F16, 128>(args, n, s) : launch_width<IO_F16, 64>(args, n, s);
  return dk == 128 ? launch_width<IO_BF16, 128>(args, n, s) : launch_width<IO_BF16, 64>(args, n, s);
}

}  // namespace lsq
