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
// 2^-160, a factor that is 0 in fp32.
//
// Precision.  The bf16 MFMA is the fast one, so every operand is a sum of
// bf16 parts: q, k and v of bf16 inputs are one part, of binary16 two, of fp32
// three (each exact), computed operands (P, S, the scaled v) are split into as
// many as their use needs, and the products of parts i + j < N are added, N = 3
// for the state and for fp32 outputs (relative 2^-24), N = 2 for 16-bit
// outputs (2^-16, against their own half step of 2^-8 or 2^-11: the outputs lose
// 2^-18 in the 2-norm, so that 0.1 to 0.3% of the bf16 and 2.4% of the binary16 ones
// are not the nearest number; with N = 3 there 0.02 and 0.07%, at 422 us instead of
// 354 for 16 prompts of 900-4096 tokens, 32 heads 128x128, and 252 instead of 224
// for one of 32768 with 16).  One rounded part instead would cost half a step of
// bf16 in the state at every chunk.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "lsq_parts.h"
#include "lsq_slots.h"
#include "lsq_slots_dev.h"

namespace lsq {
namespace dev {

// A chunk's rows of one tensor as a buffer: accesses behind its last byte read
// 0 and write nothing, so that no lane computes a clamped or 64-bit address.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* p, int64_t first, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(p)) + first, 0,
                                           bytes, 0x00027000);
}

constexpr int kCUs = 256;
constexpr int kWhole = 1024;                     // tokens that are not worth two more launches

// A lane offset behind every buffer: chunks are below 2^31 bytes.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

// Tiling of one instance: NW waves, KS of them to the same 16 value columns with
// a share of dk each; chunks of 32 tokens (one k-step of the MFMA over tokens).
template <int IO, int DK, int NW, int KS>
struct Tile {
  static constexpr int NP = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3;   // parts of an input
  static constexpr int NO = IO == IO_F32 ? 3 : 2;                       // parts on the output's side
  static constexpr int C = 32, NT = 64 * NW, DV = 16 * NW / KS, ROUND = 256;
  static constexpr int EU = IO == IO_F32 ? 4 : 8;                       // elements of a 16-byte unit
  // LDS row pitches in elements: rows 8 banks apart (P: 24), which keeps the
  // 16-byte reads of 16 rows (q, P) and the four-row reads by columns (v) free
  // of bank conflicts, and those of k, its 8-byte pieces 16 bytes apart, nearly
  // so (counters: 22% of the LDS cycles of the bf16 instance; 35% at rows 4 and
  // 20 banks apart).  P's columns are stored in the order of the k-slots: token
  // s at 8 (s % 16 / 4) + 4 (s / 16) + s % 4.
  static constexpr int PK = DK + 16, PV = DV + 16, PQ = DK + 16, PP = C + 16;
  static constexpr int QU = (C * DK / EU + NT - 1) / NT, VU = C * DV / EU / NT;   // units of k (q), v per thread
  static constexpr bool SPARE = QU * NT > C * DK / EU;                  // some threads have no unit of k
  // Two copies of the rows where two workgroups of a CU have room for them, and
  // P of two chunks (its product with v runs one chunk behind).
  static constexpr int RB = IO == IO_BF16 ? 2 : 1;
  static constexpr bool BEHIND = IO != IO_F32;
  // LDS bytes of the kernel with outputs (rows, P, the sums exchanged by two
  // waves, decays), and the workgroups of a CU, one or two at least, that its 160 KiB
  // hold: one of fp32 at Dk 128 (90 KiB), two or three of the others.  The launch
  // bounds ask for registers to match.
  static constexpr int LDS = 2 * C * (RB * NP * (PK + PV + PQ) + (BEHIND ? 2 : 1) * NO * PP) +
                             (KS > 1 ? 16 * NT : 16) + 16 * RB * ROUND;
  static constexpr int RESIDENT = 2 * LDS <= 160 * 1024 ? 2 : 1;
  static_assert(KS == 1 || (KS == 2 && !BEHIND), "the shared sums are read between the same two barriers");
};

// Four bf16 values as fp32.
__device__ __forceinline__ f32x4 widen_bf16x4(bf16x4 p) {
  const uint64_t b = __builtin_bit_cast(uint64_t, p);
  const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
  return f32x4{__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
               __uint_as_float(hi & 0xFFFF0000u)};
}

// Decays of N tokens, by token; chunk borders are every 32 tokens.
template <int N>
struct Decays {
  float hi[N], lo[N];      // L_t, the sum of log2(alpha) from the chunk's start
  float beta[N];
  float w[N];              // (c_C / c_t) beta_t
};

// x of the lane that a DPP control names, 0 where it names none or the row is
// masked out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// One wave fills the decays of its 64 tokens, two chunks, from at on (alpha 1 and
// beta 0 behind the sequence); returns the lane's log2(alpha).
template <int N>
__device__ __forceinline__ double fill_decays(Decays<N>& d, int at, float alpha, float beta, int lane) {
  double l = log2_of(alpha);
  const double own = l;
  l += dpp_or_zero<0x111, 0xF>(l);               // row_shr 1, 2, 4, 8: sums within 16 lanes
  l += dpp_or_zero<0x112, 0xF>(l);
  l += dpp_or_zero<0x114, 0xF>(l);
  l += dpp_or_zero<0x118, 0xF>(l);
  l += dpp_or_zero<0x142, 0xA>(l);               // row_bcast 15 into rows 1 and 3: within 32
  const double end = lane >= 32 ? lane_of(l, 63) : lane_of(l, 31);
  const float hi = (float)l;
  d.hi[at + lane] = hi;
  d.lo[at + lane] = (float)(l - (double)hi);
  d.beta[at + lane] = beta;
  d.w[at + lane] = exp2_of(end - l) * beta;
  return own;
}

// The first n elements of B bytes of a 16-byte unit, zeros behind them.
template <int B>
__device__ __forceinline__ u32x4 keep_elements(u32x4 x, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int in = n * B - 4 * i;                // bytes of word i that stay
    x[i] = in >= 4 ? x[i] : in <= 0 ? 0u : x[i] & 0xFFFFu;
  }
  return x;
}

// The segment a workgroup takes: sequence i, its j-th of n segments (n = 0:
// none).  With a segment length L, a sequence of more than 2 L tokens (and more
// than kWhole) is cut into its length over L, rounded up; ws is the segment's
// number among those of cut sequences, which alone use the workspace.
struct Segment {
  int i, j, n, ws;
  int64_t t0, t1;
};

__device__ __forceinline__ int segments_of(const Span& sp, int64_t L) {
  const int64_t len = sp.t1 > sp.t0 ? sp.t1 - sp.t0 : 0;
  return L == 0 || len <= 2 * L || len <= kWhole ? len > 0 : (int)((len + L - 1) / L);
}

// Segments are numbered without gaps (idle workgroups between busy ones would
// leave whole shader engines idle), 64 sequences at a time: lane r has the
// group's r-th sequence, the segments up to it and those of cut sequences among
// them.  Up to 64 sequences are ordered by length, the longest first; with more
// of them the order matters little, and a workgroup's search stays short.
struct Numbered {
  int seq, n, upto, cut;
};

__device__ __forceinline__ Numbered number_segments(const SlotArgs& a, int64_t L, int i0, int lane) {
  const bool in = i0 + lane < a.seqs;
  const Span sp = in ? span_of(a, i0 + lane) : Span{0, 0};
  const int len = sp.t1 > sp.t0 ? (int)(sp.t1 - sp.t0) : 0;
  int rank = lane;
  if (a.seqs <= 64 && in) rank = 0;              // lanes without a sequence stay behind the others
  if (a.seqs <= 64)
    for (int j = 0; j < a.seqs; ++j) {
      const int x = __builtin_amdgcn_readlane(len, j);
      rank += in && (x > len || (x == len && j < lane));
    }
  Numbered m;
  m.n = __builtin_amdgcn_ds_permute(4 * rank, segments_of(sp, L));
  m.seq = __builtin_amdgcn_ds_permute(4 * rank, i0 + lane);
  m.upto = m.n;
  m.cut = m.n > 1 ? m.n : 0;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const int up = __shfl_up(m.upto, o), cut = __shfl_up(m.cut, o);
    if (lane >= o) {
      m.upto += up;
      m.cut += cut;
    }
  }
  return m;
}

// Segment s of the batch, of the cut sequences alone where CUT.  rows:
// workgroups per segment.  PAIRED: CUs hold two workgroups.
template <bool CUT, bool PAIRED>
__device__ __forceinline__ Segment segment_of(const SlotArgs& a, int64_t L, int64_t s, int rows, int lane) {
  Segment g{};
  g.i = (int)s;
  if (L || (int64_t)a.seqs * rows > kCUs) {
    int before = 0;                              // cut segments of earlier groups
    for (int i0 = 0;; i0 += 64) {
      if (i0 >= a.seqs) return g;
      const Numbered m = number_segments(a, L, i0, lane);
      const int upto = CUT ? m.cut : m.upto, all = __builtin_amdgcn_readlane(upto, 63);
      // Where two workgroups share a CU, those of the second round come in reverse,
      // a long sequence beside a short one (16 prompts of 900-4096 tokens, 32 heads
      // 128x128 in bf16: 351 us, 369 without; fp32, 64x64: 304 and 327).  Where a CU
      // holds one, the next starts as CUs fall free, and the longest first is right
      // (fp32, 128x64: 481 us, 555 in reverse; 8 of 300-2400, 64 heads: 267 and 305).
      const int64_t round = kCUs / rows;
      if (!CUT && PAIRED && a.seqs <= 64 && s >= round && s < 2 * round && s < all)
        s = (all < 2 * round ? all : 2 * round) - 1 - (s - round);
      if (s < all) {
        const int at = __builtin_ctzll(__ballot(upto > (int)s));
        g.i = __builtin_amdgcn_readlane(m.seq, at);
        g.j = (int)s - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(m.n, at));
        g.ws = before + __builtin_amdgcn_readlane(m.cut, at) - __builtin_amdgcn_readlane(m.n, at) + g.j;
        break;
      }
      s -= all;
      before += __builtin_amdgcn_readlane(m.cut, 63);
    }
  }
  const Span sp = span_of(a, g.i);
  g.n = segments_of(sp, L);
  g.t0 = sp.t0 + (int64_t)g.j * L;
  g.t1 = g.n < 2 || g.t0 + L > sp.t1 ? sp.t1 : g.t0 + L;
  return g;
}

// Block number -> segment and row (a head's slice of value columns).  Blocks go
// to the eight XCDs in turn.  Where the rows divide by eight an XCD gets an
// eighth of them in every segment: its heads share q and k in its L2, and
// sequences of different lengths load the XCDs alike.  Segments come in order,
// so that the numbers without one are the last blocks.
struct Item {
  int64_t seg;
  int row;
};

__device__ __forceinline__ Item item_of(int64_t b, int rows) {
  if (rows % 8) return {b / rows, (int)(b % rows)};
  const int own = rows / 8;
  const int64_t p = b / 8;
  return {p / own, (int)(b % 8) * own + (int)(p % own)};
}

// One workgroup walks the chunks of one segment of one head, 16 NW / KS
// value columns of it.  Four waves compute P's tiles; every wave has its 16
// columns of S in registers in the layout that the MFMA both writes (S^T[dk, dv]
// accumulated from k^T and the scaled v) and reads (as the operand of S q): the
// k index of an operand is only a labelling, so the tiles' rows are dealt to
// the lanes as S q wants them, and in the products over tokens slots 0-3 and 4-7
// of a lane group g stand for tokens 4 g .. and 16 + 4 g ...  A chunk's
// products are independent of each other: S q and the new S, P of the same
// chunk, and (BEHIND) P v of the chunk before, with the next rows on their way
// to LDS, all between two barriers.  OUT = false adds up a segment's writes alone
// (no q, no output), for the segments behind it.  VEC: v and o by dwords and
// more (else by element: 16-bit types of odd widths or addresses).
template <int IO, int DK, int NW, int KS, bool VEC, bool OUT>
__global__ __launch_bounds__(64 * NW, (NW * Tile<IO, DK, NW, KS>::RESIDENT / 4)) void attend_kernel(AttendArgs args) {
  using T = Tile<IO, DK, NW, KS>;
  constexpr int NP = T::NP, NO = T::NO, C = T::C, PK = T::PK, PV = T::PV, PQ = T::PQ, PP = T::PP;
  constexpr int NT = T::NT, EU = T::EU, RB = T::RB, ROUND = T::ROUND, B = 16 / EU;   // B: bytes of an element
  constexpr bool BEHIND = T::BEHIND;  constexpr int CT = C / 16, DW = DK / KS, KT = DW / 16;   // a wave's part of dk
  constexpr bool AHEAD = NP == 1;                // q's operands are read a step of dk ahead (41 to 39 us at dk 64)
  constexpr int PER = NP == 1 ? 2 : 1;           // tiles of S that a step of the state's products takes
  constexpr int OT = CT / KS;                    // tiles of 16 tokens whose output a wave finishes
  const SlotArgs& a = args.s;
  __shared__ __align__(16) __bf16 kl[RB][NP][C * PK];
  __shared__ __align__(16) __bf16 vl[RB][NP][C * PV];
  __shared__ __align__(16) __bf16 ql[OUT ? RB : 1][OUT ? NP : 1][OUT ? C * PQ : 8];
  __shared__ __align__(16) __bf16 pl[OUT && BEHIND ? 2 : 1][OUT ? NO : 1][OUT ? C * PP : 8];
  __shared__ __align__(16) f32x4 part[OUT && KS > 1 ? NW * 64 : 1];
  __shared__ __align__(16) Decays<ROUND> dec[RB];
  static_assert(!OUT || sizeof(kl) + sizeof(vl) + sizeof(ql) + sizeof(pl) + sizeof(part) + sizeof(dec) == T::LDS);

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Item item = item_of(blockIdx.x, args.slices * a.heads);
  const int h = item.row / args.slices, slice = item.row % args.slices;
  const Segment sg = segment_of<!OUT, (T::RESIDENT > 1)>(a, args.seg_len, item.seg, args.slices * a.heads, lane);
  if (sg.n == 0 || (!OUT && sg.j == sg.n - 1)) return;
  // Offsets that decrease can name a token in several sequences, more of them
  // than the workspace was sized for.
  if (sg.j < 0 || sg.j >= sg.n || (sg.n > 1 && (sg.ws < 0 || sg.ws >= args.cut))) return;
  const int slot = slot_of(a, sg.i, lane);
  if (slot == kPadded) return;
  const int d0 = slice * T::DV, vcols = a.dv - d0 < T::DV ? a.dv - d0 : T::DV;   // the slice's columns
  const int64_t hk = (int64_t)(h / a.share) * DK, hv = (int64_t)h * a.dv + d0;
  if (slot == kRefused) {
    if (OUT)
      for (int64_t t = sg.t0; t < sg.t1; ++t)
        for (int c = tid; c < vcols; c += NT)
          store1<IO>(a.o, t * a.o_stride + hv + c, __uint_as_float(0x7FC00000u));
    return;
  }
  const int len = (int)(sg.t1 - sg.t0), chunks = (len + C - 1) / C;

  // ---- a chunk's rows, 16 bytes per unit, a unit's lane offset apart from its
  // neighbour's by a whole number of rows.  Rows behind the segment read as 0.
  u32x4 rq[OUT ? T::QU : 1], rk[T::QU], rv[T::VU];
  float ra = 1.f, rb = 0.f;
  constexpr int KR = NT * EU / DK, VR = NT * EU / T::DV;               // rows per pass of the threads
  const uint32_t kstep = (uint32_t)a.k_stride * B, qstep = (uint32_t)a.q_stride * B;
  const uint32_t vstep = (uint32_t)a.v_stride * B, ostep = (uint32_t)a.o_stride * B;
  const int krow = tid / (DK / EU), kcol = tid % (DK / EU) * EU, vrow = tid / (T::DV / EU), vcol = tid % (T::DV / EU) * EU;
  auto bytes_of = [&](int c, uint32_t step, uint32_t row) -> uint32_t {  // of chunk c's rows, 0 behind the last
    const int live = len - c * C < C ? len - c * C : C;
    return live > 0 ? (uint32_t)(live - 1) * step + row : 0u;
  };
  // A round of decays: one token per thread of the last four waves, read a round
  // ahead.
  const int dtok = tid - (NT - ROUND);
  auto read_decays = [&](int t) {
    if (dtok < 0) return;
    const int64_t x = (sg.t0 + (t + dtok < len ? t + dtok : len - 1)) * a.heads + h;
    ra = a.alpha[x];
    rb = a.beta[x];
  };
  double total = 0.0;
  auto put_decays = [&](int t, int buf) {
    if (dtok >= 0) {
      const bool in = t + dtok < len;
      total += fill_decays(dec[buf], dtok & ~63, in ? ra : 1.f, in ? rb : 0.f, lane);
    }
  };
  auto read_chunk = [&](int c) {
    const int64_t t = sg.t0 + c * C;
    const auto kb = rows_of(a.k, (t * a.k_stride + hk) * B, bytes_of(c, kstep, DK * B));
    const auto qb = rows_of(a.q, (t * a.q_stride + hk) * B, bytes_of(c, qstep, DK * B));
    const auto vb = rows_of(a.v, (t * a.v_stride + hv) * B, bytes_of(c, vstep, vcols * B));
    uint32_t ko = krow * kstep + kcol * B, qo = krow * qstep + kcol * B, vo = vrow * vstep + vcol * B;
#pragma unroll
    for (int n = 0; n < T::QU; ++n) {
      rk[n] = __builtin_amdgcn_raw_buffer_load_b128(kb, ko, 0, 0);
      ko += KR * kstep;
      if constexpr (OUT) rq[n] = __builtin_amdgcn_raw_buffer_load_b128(qb, qo, 0, 0);
      qo += KR * qstep;
    }
#pragma unroll
    for (int n = 0; n < T::VU; ++n) {
      if constexpr (VEC) {
        rv[n] = __builtin_amdgcn_raw_buffer_load_b128(vb, vo, 0, 0);
      } else {
        uint32_t w[EU];
#pragma unroll
        for (int x = 0; x < EU; ++x) w[x] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(vb, vo + x * B, 0, 0);
#pragma unroll
        for (int x = 0; x < EU / 2; ++x) rv[n][x] = w[2 * x] | w[2 * x + 1] << 16;
      }
      vo += VR * vstep;
    }
  };
  auto put = [&](u32x4 r, auto* dst, int row, int pitch, int col) {   // one unit's parts
    __bf16* p = &dst[0][row * pitch + col];
    constexpr int plane = sizeof(dst[0]) / sizeof(__bf16);
    if constexpr (IO == IO_BF16) {
      *reinterpret_cast<u32x4*>(p) = r;
    } else if constexpr (IO == IO_F32) {
      bf16x4 s[NP];
      split4<NP>(__builtin_bit_cast(f32x4, r), s);
#pragma unroll
      for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x4*>(p + i * plane) = s[i];
    } else {
      bf16x4 s[2][NP];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = __half2float(__ushort_as_half((unsigned short)(r[2 * y + e / 2] >> (16 * (e & 1)))));
        split4<NP>(x, s[y]);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x8*>(p + i * plane) = join(s[0][i], s[1][i]);
    }
  };
  // Rows closer than their own length (a broadcast input) do not read as 0
  // behind the segment, nor do columns behind dv.
  const bool overlap = kstep < DK * B || qstep < DK * B || vstep < (uint32_t)vcols * B;
  auto put_chunk = [&](int c, int buf) {
    if (overlap && len - c * C < C) {
      const u32x4 zero = {0, 0, 0, 0};
      const int live = len - c * C;
#pragma unroll
      for (int n = 0; n < T::QU; ++n)
        if (n * KR + krow >= live) {
          rk[n] = zero;
          if constexpr (OUT) rq[n] = zero;
        }
#pragma unroll
      for (int n = 0; n < T::VU; ++n)
        if (n * VR + vrow >= live) rv[n] = zero;
    }
    if (vcols < T::DV) {
#pragma unroll
      for (int n = 0; n < T::VU; ++n) rv[n] = keep_elements<B>(rv[n], vcols - vcol);
    }
#pragma unroll
    for (int n = 0; n < T::QU; ++n)
      if (!T::SPARE || n * KR + krow < C) {
        put(rk[n], kl[buf], n * KR + krow, PK, kcol);
        if constexpr (OUT) put(rq[n], ql[buf], n * KR + krow, PQ, kcol);
      }
#pragma unroll
    for (int n = 0; n < T::VU; ++n) put(rv[n], vl[buf], n * VR + vrow, PV, vcol);
  };

  // ---- the state's columns: lane li has column li of the wave's 16, and of
  // S^T the rows 32 (I / 2) + 8 g + 4 (I % 2) + v (tiles I = 2 m and 2 m + 1
  // together hold eight consecutive rows per lane, an operand's k-slots)
  const int w0 = 16 * (wave / KS), kh = wave % KS;   // the wave's first column in the slice; its part of dk
  f32x4 S[KT];
  const int64_t state = ((int64_t)h * a.dv + d0 + w0 + li) * DK + kh * DW + 8 * g, per = (int64_t)a.heads * a.dv * DK;
  float* slot_S = a.S + slot * per + state;
  float* seg_S = args.ws + sg.ws * per + state;
  {
    const bool from_ws = OUT && sg.n > 1;
    const bool zero = !OUT || (!from_ws && a.fresh && a.fresh[sg.i]);
    const float* p = from_ws ? seg_S : slot_S;
#pragma unroll
    for (int I = 0; I < KT; ++I)
      S[I] = !zero && w0 + li < vcols ? *reinterpret_cast<const f32x4*>(p + 32 * (I / 2) + 4 * (I % 2))
                                      : f32x4{0.f, 0.f, 0.f, 0.f};
  }

  bf16x4 vr[2][NP];                              // the wave's columns of v, by columns
  f32x4 acc[OUT ? CT : 1];                       // o^T tiles: rows dv, columns t (KS = 2: only tile 0 once the halves are exchanged)
  // A v that is not finite may reach its own column from its token on, but P's
  // zeros times it would be NaN for the chunk's earlier tokens too.  It has made
  // its column of the new S NaN, so one register of S tells (a look at all of v
  // would be ten instructions per chunk): such a v becomes 0 in P v, and the
  // column's outputs NaN from it on.  While S is finite the branch costs 1%
  // (16 x 2560 tokens of 32 heads 128x128 in bf16: 326 us without, 330 with).
  auto keep_causal = [&]() __attribute__((always_inline)) {
    int first = C;                               // of column li
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((__builtin_bit_cast(uint64_t, vr[y][0]) >> (16 * e) & 0x7F80) == 0x7F80) {
          const int t = 16 * y + 4 * g + e;
          first = t < first ? t : first;
#pragma unroll
          for (int i = 0; i < NP; ++i) vr[y][i][e] = (__bf16)0.f;
        }
    }
    for (int o = 16; o < 64; o *= 2) {
      const int other = __shfl_xor(first, o);
      first = other < first ? other : first;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int from = __shfl(first, 4 * g + v);
#pragma unroll
      for (int ti = 0; ti < OT; ++ti)
        if ((KS > 1 ? 16 * kh : 16 * ti) + li >= from) acc[ti][v] = __uint_as_float(0x7FC00000u);
    }
  };
  // acc += P v of a chunk, rounded
  using Out = typename std::conditional<IO == IO_F32, f32x4, u32x2>::type;   // four columns of a token
  Out out[OUT ? OT : 1];
  const int t0 = KS > 1 ? 16 * kh : 0;           // the wave's first token
  auto finish = [&](int buf) __attribute__((always_inline)) {
    if (__builtin_expect(__any(S[0][0] != S[0][0]), 0)) keep_causal();
    if constexpr (KS > 1) acc[0] = acc[0] + part[wave * 64 + lane];
#pragma unroll
    for (int ti = 0; ti < OT; ++ti) {
      bf16x8 pp[NO];
#pragma unroll
      for (int i = 0; i < NO; ++i) {
        pp[i] = *reinterpret_cast<const bf16x8*>(&pl[buf][i][(t0 + 16 * ti + li) * PP + 8 * g]);
      }
#pragma unroll
      for (int i = NO - 1; i >= 0; --i)          // small products first
#pragma unroll
        for (int j = NP - 1; j >= 0; --j)
          if (i + j < NO) acc[ti] = mfma(join(vr[0][j], vr[1][j]), pp[i], acc[ti]);
    }
#pragma unroll
    for (int ti = 0; ti < OT; ++ti) {
      const f32x4 x = acc[ti];
      if constexpr (IO == IO_F32) out[ti] = x;
      else out[ti] = u32x2{pair16<IO>(x[0], x[1]), pair16<IO>(x[2], x[3])};
    }
  };
  // Chunk c's outputs to memory.  A wait for loads counts the stores issued
  // behind them too, so the one-copy instances store where no load is in flight
  // that is waited for soon (4 prompts of 650-2500 tokens, 64 heads 128x64 in
  // fp32: 211 us; 223 with the stores before the put of the next rows).  With
  // two copies it makes no difference.
  auto store_out = [&](int c) __attribute__((always_inline)) {
    const auto ob = rows_of(a.o, ((sg.t0 + c * C) * a.o_stride + hv) * B, c < 0 ? 0u : bytes_of(c, ostep, vcols * B));
    uint32_t oo = (t0 + li) * ostep + (w0 + 4 * g) * B;
    const int left = vcols - (w0 + 4 * g);       // columns to write, four per lane
#pragma unroll
    for (int ti = 0; ti < OT; ++ti) {
      const Out x = out[ti];
      if (VEC && vcols % 4 == 0) {
        const uint32_t e = left > 0 ? oo : kNowhere;
        if constexpr (IO == IO_F32)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), ob, e, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b64(x, ob, e, 0, 0);
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const uint32_t e = v < left ? oo + v * B : kNowhere;
          if constexpr (IO == IO_F32)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[v]), ob, e, 0, 0);
          else if constexpr (!VEC)
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(x[v / 2] >> (16 * (v & 1))), ob, e, 0, 0);
          else if (v % 2 == 0)
            __builtin_amdgcn_raw_buffer_store_b32(x[v / 2], ob, e, 0, 0);
        }
      }
      oo += 16 * ostep;
    }
  };

  read_decays(0);
  read_chunk(0);
  put_decays(0, 0);
  put_chunk(0, 0);
  if constexpr (RB == 2) read_chunk(1);
#pragma unroll
  for (int ti = 0; ti < (OUT ? CT : 1); ++ti) acc[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int y = 0; y < 2; ++y)
#pragma unroll
    for (int i = 0; i < NP; ++i) vr[y][i] = bf16x4{};
  for (int c = 0; c < chunks; ++c) {
    const int buf = RB == 2 ? c & 1 : 0, at = c * C % ROUND;
    const Decays<ROUND>& d = dec[RB == 2 ? c / (ROUND / C) & 1 : 0];
    __syncthreads();
    if constexpr (OUT && BEHIND) {
      finish((c & 1) ^ 1);
      if constexpr (RB == 2) store_out(c - 1);
    }
    if constexpr (OUT) {
      // ---- P^T tile of a wave: rows s, columns t; the tile above the diagonal is 0
      // and put once into each buffer
      if ((NW == 4 || wave < 4) && (wave != 1 || c < 2)) {
        const int ti = wave >> 1, si = wave & 1;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) {
          bf16x8 kp[NP], qp[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            kp[i] = *reinterpret_cast<const bf16x8*>(&kl[buf][i][(16 * si + li) * PK + 32 * ks + 8 * g]);
            qp[i] = *reinterpret_cast<const bf16x8*>(&ql[buf][i][(16 * ti + li) * PQ + 32 * ks + 8 * g]);
          }
#pragma unroll
          for (int i = NP - 1; i >= 0; --i)
#pragma unroll
            for (int j = NP - 1; j >= 0; --j)
              if (i + j < NO) x = mfma(kp[i], qp[j], x);
        }
        const int t = 16 * ti + li, s0 = 16 * si + 4 * g;
        const float ht = d.hi[at + t], lt = d.lo[at + t];
        const f32x4 hs = *reinterpret_cast<const f32x4*>(&d.hi[at + s0]), ls = *reinterpret_cast<const f32x4*>(&d.lo[at + s0]);
        const f32x4 bs = *reinterpret_cast<const f32x4*>(&d.beta[at + s0]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float y = x[v] * (__builtin_amdgcn_exp2f((ht - hs[v]) + (lt - ls[v])) * bs[v]);
          x[v] = s0 + v <= t ? y : 0.f;
        }
        bf16x4 parts[NO];
        split4<NO>(x, parts);
#pragma unroll
        for (int i = 0; i < NO; ++i) *reinterpret_cast<bf16x4*>(&pl[BEHIND ? c & 1 : 0][i][t * PP + 8 * g + 4 * si]) = parts[i];
      }
      if constexpr (RB == 2) __builtin_amdgcn_s_setprio(1);
      // ---- c_t S q
      bf16x8 qp[2][CT][NP];
      auto read_q = [&](int ks) __attribute__((always_inline)) {
#pragma unroll
        for (int ti = 0; ti < CT; ++ti)
#pragma unroll
          for (int i = 0; i < NP; ++i)
            qp[ks & 1][ti][i] = *reinterpret_cast<const bf16x8*>(&ql[buf][i][(16 * ti + li) * PQ + kh * DW + 32 * ks + 8 * g]);
      };
      if constexpr (AHEAD) read_q(0);
#pragma unroll
      for (int ks = 0; ks < DW / 32; ++ks) {
        bf16x8 sp[NO];
        bf16x4 s0[NO], s1[NO];
        split4<NO>(S[2 * ks], s0);
        split4<NO>(S[2 * ks + 1], s1);
#pragma unroll
        for (int i = 0; i < NO; ++i) sp[i] = join(s0[i], s1[i]);
        if constexpr (!AHEAD) {
          read_q(ks);
        } else if (ks + 1 < DW / 32) {
          read_q(ks + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int ti = 0; ti < CT; ++ti) {
#pragma unroll
          for (int i = NO - 1; i >= 0; --i)
#pragma unroll
            for (int j = NP - 1; j >= 0; --j)
              if (i + j < NO)
                acc[ti] = mfma(sp[i], qp[ks & 1][ti][j], ks == 0 && i == NO - 1 && j == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[ti]);
        }
      }
#pragma unroll
      for (int ti = 0; ti < CT; ++ti) {
        const float ct = __builtin_amdgcn_exp2f(d.hi[at + 16 * ti + li]) * (1.f + 0.69314718f * d.lo[at + 16 * ti + li]);
        acc[ti] = acc[ti] * ct;
      }
      if constexpr (KS > 1) {                    // the other wave's tile to it, the own one to place 0
        part[(wave ^ 1) * 64 + lane] = kh ? acc[0] : acc[1];
        acc[0] = kh ? acc[1] : acc[0];
      }
    }
    if constexpr (RB == 1) {
      if constexpr (OUT && BEHIND) store_out(c - 1);
      if (c + 1 < chunks) read_chunk(c + 1);
    }
    const bool round = at + C == ROUND;          // the next chunk opens a round of decays
    if constexpr (RB == 2) {
      // rows of c + 1 to LDS, of c + 2 from memory; the decays between them, where
      // no younger load is in flight that their wait would include
      put_chunk(c + 1, buf ^ 1);
      if (round && c + 1 < chunks) put_decays((c + 1) * C, ((c + 1) / (ROUND / C)) & 1);
      if (at == 0) read_decays(c * C + ROUND);
      read_chunk(c + 2);
    }
    if constexpr (RB == 2) __builtin_amdgcn_s_setprio(2);
    // ---- S = c_C S + k^T (w v); one part: PER tiles at a time, the next ones'
    // operands read before their products (1000 tokens of 4 heads 128x128 in
    // bf16: 65 us; 69 one by one).  More parts have products enough to wait
    // behind, and no registers to spare (binary16: 90 us one by one, 119 so).
    bf16x8 vs[3];
    bf16x4 half[2][3];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int i = 0; i < NP; ++i)
        vr[y][i] = read_column4(&vl[buf][i][(16 * y + 4 * g + li / 4) * PV + w0 + 4 * (li % 4)]);
      f32x4 x = widen_bf16x4(vr[y][0]);
#pragma unroll
      for (int i = 1; i < NP; ++i) x = x + widen_bf16x4(vr[y][i]);
      x = x * *reinterpret_cast<const f32x4*>(&d.w[at + 16 * y + 4 * g]);
      split4<3>(x, half[y]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) vs[i] = join(half[0][i], half[1][i]);
    const float gamma = __builtin_amdgcn_exp2f(d.hi[at + C - 1]) * (1.f + 0.69314718f * d.lo[at + C - 1]);   // c_C
    bf16x8 kp[2][PER][NP];
    auto read_k = [&](int m) __attribute__((always_inline)) {
#pragma unroll
      for (int y = 0; y < PER; ++y)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int I = PER * m + y;
          const __bf16* p = &kl[buf][i][(4 * g + li / 4) * PK + kh * DW + 32 * (I / 2) + 8 * (li % 4) + 4 * (I % 2)];
          kp[m & 1][y][i] = join(read_column4(p), read_column4(p + 16 * PK));
        }
    };
    if constexpr (PER > 1) read_k(0);
#pragma unroll
    for (int m = 0; m < KT / PER; ++m) {
      if constexpr (PER == 1) {
        read_k(m);
      } else if (m + 1 < KT / PER) {
        read_k(m + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int y = 0; y < PER; ++y) S[PER * m + y] = S[PER * m + y] * gamma;
#pragma unroll
      for (int i = NP - 1; i >= 0; --i)
#pragma unroll
        for (int j = 2; j >= 0; --j)
          if (i + j < 3)
#pragma unroll
            for (int y = 0; y < PER; ++y) S[PER * m + y] = mfma(kp[m & 1][y][i], vs[j], S[PER * m + y]);
    }
    if constexpr (RB == 2) __builtin_amdgcn_s_setprio(0);
    if constexpr (RB == 1) {
      __syncthreads();
      if constexpr (OUT && !BEHIND) finish(0);
      if (c + 1 < chunks) {
        put_chunk(c + 1, 0);
        if (round) put_decays((c + 1) * C, 0);
        if (at == 0) read_decays(c * C + ROUND);
      }
      if constexpr (OUT && !BEHIND) store_out(c);
    }
  }
  if constexpr (OUT && BEHIND) {
    __syncthreads();
    finish((chunks - 1) & 1);
    store_out(chunks - 1);
  }

  if (!OUT || sg.j == sg.n - 1) {
    float* p = OUT ? slot_S : seg_S;
    if (w0 + li < vcols) {
#pragma unroll
      for (int I = 0; I < KT; ++I) *reinterpret_cast<f32x4*>(p + 32 * (I / 2) + 4 * (I % 2)) = S[I];
    }
  }
  if constexpr (!OUT) {                          // the segment's own decay
    __shared__ double sum[NW];
#pragma unroll
    for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
    if (lane == 0) sum[wave] = total;
    __syncthreads();
    if (slice == 0 && tid == 0) {
      for (int w = 1; w < NW; ++w) total += sum[w];
      args.ws_decay[sg.ws * a.heads + h] = exp2_of(total);
    }
  }
}

// The states before each segment of a sequence of several: S_0 is the slot's
// (or 0), S_{j+1} = decay_j S_j + writes_j; segment j's writes are replaced by
// S_j.  A thread takes four elements through all the segments.
__global__ __launch_bounds__(256) void combine_kernel(AttendArgs args, int blocks, int64_t quads) {
  const SlotArgs& a = args.s;
  const int b = blockIdx.x % blocks, i = blockIdx.x / blocks;
  const Span sp = span_of(a, i);
  const int n = segments_of(sp, args.seg_len);
  if (n < 2) return;
  const int lane = threadIdx.x & 63, slot = slot_of(a, i, lane);
  if (slot < 0) return;
  int64_t first = 0;                             // the sequence's first segment in the workspace
  for (int i0 = 0;; i0 += 64) {
    const Numbered m = number_segments(a, args.seg_len, i0, lane);
    if (i < i0 + 64) {
      first += __builtin_amdgcn_readlane(m.cut, __builtin_ctzll(__ballot(m.seq == i))) - n;
      break;
    }
    first += __builtin_amdgcn_readlane(m.cut, 63);
  }
  if (first < 0 || first + n > args.cut) return;   // decreasing offsets, as above
  const int64_t per_head = quads / a.heads;
  const bool fresh = a.fresh && a.fresh[i];
  for (int64_t q = (int64_t)b * 256 + threadIdx.x; q < quads; q += (int64_t)blocks * 256) {
    const float* decay = args.ws_decay + first * a.heads + q / per_head;
    f32x4 S = {0.f, 0.f, 0.f, 0.f};
    if (!fresh) S = reinterpret_cast<const f32x4*>(a.S)[slot * quads + q];
    f32x4* ws = reinterpret_cast<f32x4*>(args.ws) + first * quads + q;
    for (int j0 = 0; j0 < n; j0 += 4) {          // four segments' writes in flight
      f32x4 x[4];
      float c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = j0 + j < n - 1 ? j0 + j : n - 2;   // the last segment's writes are not needed
        x[j] = ws[k * quads];
        c[j] = decay[k * a.heads];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j < n) {
          ws[(j0 + j) * quads] = S;
          S = S * c[j] + x[j];
        }
    }
  }
}

}  // namespace dev

namespace {

// Value columns of a workgroup.  Three bf16 parts of fp32 rows take 66 KiB of LDS
// at 64 columns of Dk 64, 90 at Dk 128.
int slice_width(int io, int dv) { return io == IO_F32 || dv <= 64 ? 64 : 128; }

template <int IO, int DK, int NW, int KS, bool VEC>
hipError_t launch_instance(const AttendArgs& args, hipStream_t s) {
  const SlotArgs& a = args.s;
  const int64_t rows = (int64_t)args.slices * a.heads, blocks = args.segments * rows, cut = args.cut * rows;
  const int64_t quads = (int64_t)a.heads * a.dv * DK / 4, most = 4096 / a.seqs + 1;
  const int64_t per = (quads + 255) / 256 < most ? (quads + 255) / 256 : most;
  if (!fits_launch(blocks, 64 * NW) ||
      (args.seg_len && (!fits_launch(cut, 64 * NW) || !fits_launch(per * a.seqs, 256))))
    return hipErrorInvalidConfiguration;
  if (args.seg_len) {
    hipLaunchKernelGGL((dev::attend_kernel<IO, DK, NW, KS, VEC, false>), dim3((unsigned)cut), dim3(64 * NW), 0, s, args);
    hipLaunchKernelGGL(dev::combine_kernel, dim3((unsigned)(per * a.seqs)), dim3(256), 0, s, args,
                       (int)per, quads);
  }
  hipLaunchKernelGGL((dev::attend_kernel<IO, DK, NW, KS, VEC, true>), dim3((unsigned)blocks), dim3(64 * NW), 0, s, args);
  return hipGetLastError();
}

template <int IO, int DK>
hipError_t launch_width(const AttendArgs& args, hipStream_t s) {
  if constexpr (IO == IO_F32) {
    return launch_instance<IO, DK, 8, 2, true>(args, s);
  } else {
    if (slice_width(IO, args.s.dv) == 128)
      return args.wide ? launch_instance<IO, DK, 8, 1, true>(args, s)
                       : launch_instance<IO, DK, 8, 1, false>(args, s);
    return args.wide ? launch_instance<IO, DK, 4, 1, true>(args, s)
                     : launch_instance<IO, DK, 4, 1, false>(args, s);
  }
}

}  // namespace

AttendPlan attend_plan(int64_t tokens, int32_t seqs, int32_t heads, int32_t dk, int32_t dv, int io) {
  AttendPlan p{};
  const int width = slice_width(io, dv);
  p.slices = (dv + width - 1) / width;
  p.segments = seqs;
  // A segment: a 512th of the work (two workgroups on each of 256 CUs; for fp32 at
  // Dk 128 one after the other), but 256 tokens at least, and more where a long
  // sequence has few rows, so that the combination's steps (0.5 us each) and a
  // segment's chunks (3.5 us for both passes) take as long.  The host does not see the lengths: where the rows
  // alone occupy the CUs, or the sequences are short on average, a batch of few
  // tokens is taken whole; otherwise the kernels cut the sequences of more than
  // two segments.
  const int64_t rows = (int64_t)heads * p.slices;
  int64_t L = tokens * rows / 512;
  const int64_t root = (int64_t)(2.0 * sqrt((double)tokens));
  if (L < root) L = root;
  if (L < 256) L = 256;
  L = (L + 63) / 64 * 64;
  const bool alone = (int64_t)seqs * rows < dev::kCUs && tokens >= (int64_t)seqs * dev::kWhole;
  if (tokens > dev::kWhole && (alone || tokens >= (8 * L > 4096 ? 8 * L : 4096))) {
    p.seg_len = L;
    p.segments = tokens / L + seqs;
    // a cut sequence has more than 2 L tokens and at most one segment that is
    // not full: fewer than half as many again as there are full ones
    p.cut = tokens / L + tokens / (2 * L) + 1;
    p.state_bytes = p.cut * heads * dv * dk * 4;
    p.workspace = (size_t)(p.state_bytes + p.cut * heads * 4);
  }
  return p;
}

hipError_t launch_attend(const AttendArgs& args, int io, int dk, hipStream_t s) {
  if (io == IO_F32) return dk == 128 ? launch_width<IO_F32, 128>(args, s) : launch_width<IO_F32, 64>(args, s);
  if (io == IO_F16) return dk == 128 ? launch_width<IO_F16, 128>(args, s) : launch_width<IO_F16, 64>(args, s);
  return dk == 128 ? launch_width<IO_BF16, 128>(args, s) : launch_width<IO_BF16, 64>(args, s);
}

}  // namespace lsq
