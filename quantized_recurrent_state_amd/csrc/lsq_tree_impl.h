// Trees of drafted tokens over the slots of an fp32 handle: the recurrence along
// every path, the slots left as they are.  Instantiated per input type in
// lsq_tree_*.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "lsq_parts.h"
#include "lsq_slots.h"
#include "lsq_slots_dev.h"
#include "lsq_step_impl.h"

namespace lsq {
namespace dev {

// Nodes on the way from each lane's node to its root, itself included, as a bit
// mask, from the lanes' parents (-1 above a root), and the sums of x along the same
// ways: by pointer doubling, as many rounds as the depth has bits.
template <bool SUM>
__device__ __forceinline__ uint64_t path_mask(int parent, int lane, double& x) {
  uint64_t mask = (uint64_t)1 << lane;
  int up = parent;
  while (__any(up >= 0)) {
    const int at = up < 0 ? lane : up;
    const uint32_t lo = __shfl((int)(uint32_t)mask, at), hi = __shfl((int)(uint32_t)(mask >> 32), at);
    const double add = SUM ? __shfl(x, at) : 0.0;
    const int next = __shfl(up, at);
    mask |= (uint64_t)hi << 32 | lo;
    if (up >= 0) {
      if constexpr (SUM) x += add;
      up = next;
    }
  }
  return mask;
}

// The trees on the matrix cores.  With g_j the product of the decays on node
// j's path and D_ij of those behind i up to j,
//   w_j = beta_j (v_j - delta (g_j S k_j + sum_{i above j} D_ij (k_i.k_j) w_i))
//   o_j = g_j S q_j + sum_{i above j, and j} D_ij (k_i.q_j) w_i,
// so the state is read once for all nodes and no node's state is formed.
//   S k, S q  [nodes x dv], the products with the state: node rows from LDS, the
//             state's rows straight from memory in the operand's layout;
//   P, M      [nodes x nodes], D_ij (k_i.q_j) and D_ij (k_i.k_j) on the paths, 0 elsewhere;
//   w         16 nodes at a time: earlier tiles by products with M, the tile itself by
//             T = (I + diag(beta) M)^-1 of its 16 x 16 block;
//   o         P w on top of g S q.
// A wave has 16 value columns from the state to the output; P, M and T are made
// once per workgroup.  Under a scalar decay D is 2^(L_j - L_i), L the sums of log2
// of the decays along the paths (fp64, held as two floats), with the sign of
// the negative ones between; under a diagonal one P and M are summed on the way up
// from each node, which leaves g_j k_j and g_j q_j for the products with S.
//
// Precision: every operand that is not an input is a sum of three bf16 parts (24 bits)
// and the products of parts i + j < 3 are added, so that outputs of every type have
// fp32's accuracy before their one rounding.  (Two parts for the 16-bit types missed up
// to 2^-16 of the terms where these cancel, and took 35 us instead of 36 for the 64 trees
// below, 26 instead of 28 for the 32 and 105 instead of 108 for the 256.)
//
// What is not finite would reach other paths through the zeros of P, M and T.  A
// w that is not, before or behind T, counts as 0, and the outputs behind its node in its
// column become NaN; a row of T that is not counts as 0 and spoils all columns so.
//
// Bound by the state's bytes where there are many trees (256 of 8 nodes, 32 heads of
// 128x128 in bf16 with the delta rule: 108 us, 5.4 TB/s of state and rows), by rounds of
// workgroups whose loads and products take turns where there are few (64 of 6-16
// nodes: 36 us, 4.3 TB/s; 32 of 40-64, 64 heads 128x64, linear write: 27-28 us).  The loads
// and stores alone took 107, 31 and 29 us in these workgroups.
template <int IO, int DK, int DELTA, int DIAG, int NT, int NW>
struct TreeTile {
  static constexpr int IN = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3;   // parts of an input
  static constexpr int NO = 3, NR = DIAG ? NO : IN;                     // of what is computed, of the node rows
  static constexpr int N = 16 * NT, W = (N + 31) / 32 * 32;             // nodes; columns of P and M as parts
  // Pitches in elements: node rows, P and M as parts and as fp32, T, rows of the walk.
  // (Those of P and M decide how many workgroups a CU holds: with W + 16 the 32 trees
  // above take 31 us.)
  static constexpr int PK = DK + 16, PW = W + 8, PP = N + 4, PT = 20, PR = DK + 4;
  static constexpr int EU = IO == IO_F32 ? 4 : 8;                       // elements of a 16-byte unit
  static constexpr int UNITS = (N * DK / EU + 64 * NW - 1) / (64 * NW); // units of q (k) per thread
  static constexpr int ROUNDS = (4 * NT + NW - 1) / NW;                 // nodes a lane group walks up from
  // Tiles of P, with the zeros behind the diagonal in a pair of them, and of M behind
  // the first row of tiles.
  static constexpr int PTILES = NT == 1 ? 2 : NT == 2 ? 4 : NT == 3 ? 8 : 12;
  static constexpr int MTILES = !DELTA || NT == 1 ? 0 : NT == 2 ? 2 : NT == 3 ? 4 : 8;
  static constexpr int TASKS = (PTILES + MTILES + NW - 1) / NW;
  // 16-bit rows of v come, and of o go, through LDS: value columns of all waves, whole
  // 128-byte lines instead of 32-byte pieces.
  static constexpr bool STAGED = IO != IO_F32;
  static constexpr int C = 16 * NW, PC = C + 8, VUNITS = (N * C / 8 + 64 * NW - 1) / (64 * NW);
  // LDS, in bytes.  P and M as parts, and the rows of v, take the place of the node
  // rows once the products with S are done; one tile's have room beside them, and a
  // diagonal decay's rows of v of two.
  static constexpr bool OVERLAY = NT > 1 && !DIAG, LATE = OVERLAY || (DIAG && DELTA && NT > 2);
  static constexpr int max2(int x, int y) { return x > y ? x : y; }
  static constexpr int ROWS = 2 * NR * N * PK * (DIAG && !DELTA ? 1 : 2);
  static constexpr int PARTS = DIAG ? 0 : 2 * PW * NO * N * (MTILES ? 2 : 1) - (MTILES ? 32 * PW : 0);
  static constexpr int VROWS = STAGED ? 2 * N * PC : 0;
  static constexpr int RAW = DIAG ? 8 * N * PR : 0;
  static constexpr int PARTS_AT = OVERLAY ? 0 : ROWS, VROWS_AT = LATE && DIAG ? 0 : PARTS_AT + (DIAG ? max2(0, RAW - ROWS) : PARTS);
  static constexpr int P_AT = max2(max2(ROWS, RAW), VROWS_AT + VROWS);  // P in fp32
  // M in fp32, or its diagonal blocks: behind the node rows, in the place of its parts.
  static constexpr int M_AT = OVERLAY ? ROWS : P_AT + (DIAG ? 4 * N * PP : 0);
  static constexpr int M = !DELTA ? 0 : DIAG ? 4 * N * PP : 64 * NT * PT;
  static constexpr int T_AT = max2(P_AT, M_AT + M);
  static constexpr int BYTES = T_AT + (DELTA ? 2 * NO * N * PT : 0);
};

// What all waves of a workgroup know of the nodes.
struct TreeNodes {
  float hi[64], lo[64], g[64], beta[64];         // L, 2^L with its sign, beta
  uint32_t on[2][64];                            // the paths, by 32 nodes
  uint64_t neg;                                  // nodes with a negative decay
  unsigned long long spoilt;                     // whose row of T is not finite
};

// What rounds to infinity as a bf16 part, from here on, counts as not finite.
constexpr float kLargest = 0x1.ffp127f;

template <int N, int NA, int NB>
__device__ __forceinline__ f32x4 mfma_parts(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
  for (int x = NA - 1; x >= 0; --x)              // the small products first
#pragma unroll
    for (int y = NB - 1; y >= 0; --y)
      if (x + y < N) c = mfma(a[x], b[y], c);
  return c;
}

// Where element c of a row lies: the k-slots of lane group g hold elements
// 4 g .. 4 g + 3 of both halves of each 32, so that a 16-byte load of the state
// by every lane takes whole 64-byte runs of its rows.
__device__ __forceinline__ int slot_order(int c) { return (c & ~31) + 8 * ((c & 15) >> 2) + ((c & 16) >> 2) + (c & 3); }

// x as P parts to the planes of an array.
template <int P>
__device__ __forceinline__ void put4(__bf16* dst, int plane, f32x4 x) {
  bf16x4 p[P];
  split4<P>(x, p);
#pragma unroll
  for (int y = 0; y < P; ++y) *reinterpret_cast<bf16x4*>(dst + y * plane) = p[y];
}

template <int P>
__device__ __forceinline__ void get8(const __bf16* src, int plane, bf16x8 (&out)[P]) {
#pragma unroll
  for (int y = 0; y < P; ++y) out[y] = *reinterpret_cast<const bf16x8*>(src + y * plane);
}

// One head of a tree of up to 16 NT nodes, more than 16 (NT - 1).
template <int IO, int DK, int DELTA, int DIAG, int NT, int NW>
__device__ __forceinline__ void tree_head(const TreeArgs& a, char* lds, TreeNodes& nl, int i, int h, int rb, int slot,
                                          int64_t t0, int n) {
  using T = TreeTile<IO, DK, DELTA, DIAG, NT, NW>;
  constexpr int N = T::N, PK = T::PK, PP = T::PP, PW = T::PW, PT = T::PT, PR = T::PR, KS = DK / 32, NO = T::NO, NR = T::NR;
  constexpr int kRow = N * PK, kPart = N * PW, kT = N * PT;            // planes
  __bf16* const ql = reinterpret_cast<__bf16*>(lds);
  __bf16* const kl = ql + NR * kRow;
  __bf16* const pp = reinterpret_cast<__bf16*>(lds + T::PARTS_AT);     // P, then M, as parts
  __bf16* const mp = pp + NO * kPart - 16 * PW;                        // M has no first row of tiles
  uint16_t* const vl = reinterpret_cast<uint16_t*>(lds + T::VROWS_AT);
  float* const pl = reinterpret_cast<float*>(lds + T::P_AT);
  float* const ml = reinterpret_cast<float*>(lds + T::M_AT);
  __bf16* const tl = reinterpret_cast<__bf16*>(lds + T::T_AT);

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const SlotArgs& b = a.s;
  const int row0 = (rb * NW + wave) * 16, row = row0 + lc;   // the lane's value column
  const int rowc = row < b.dv ? row : b.dv - 1;
  const int hk = h / b.share * DK;
  const int64_t hv = (int64_t)h * b.dv;
  // Element offset of node j's row; rows behind the last repeat it.
  auto at_node = [&](int j, int64_t stride) { return (uint64_t)(uint32_t)(j < n ? j : n - 1) * (uint32_t)stride; };
  auto behind = [](const void* p, int64_t e) { return static_cast<const typename Raw<IO>::One*>(p) + e; };
  const auto* const kb = behind(b.k, t0 * b.k_stride + hk);
  const auto* const qb = behind(b.q, t0 * b.q_stride + hk);
  const auto* const vb = behind(b.v, t0 * b.v_stride + hv);
  const float* const ab = b.alpha + (t0 * b.heads + h) * (DIAG ? DK : 1);

  // ---- loads, in the order of their use: node rows, v, the state
  int parent = lane < n ? a.parents[t0 + lane] : -1;
  constexpr int EU = T::EU, ROWU = DK / EU;      // units of a row
  auto unit_in = [&](int x) { return (x + 1) * 64 * NW <= N * ROWU || x * 64 * NW + tid < N * ROWU; };
  u32x4 rq[DIAG ? 1 : T::UNITS], rk[T::UNITS];
  float4 rd[DIAG ? T::UNITS : 1][EU / 4];
#pragma unroll
  for (int x = 0; x < T::UNITS; ++x) {
    const int u = x * 64 * NW + tid, j = u / ROWU, c = u % ROWU * EU;
    if (unit_in(x)) {
      rk[x] = *reinterpret_cast<const u32x4*>(kb + at_node(j, b.k_stride) + c);
      if constexpr (DIAG) {
#pragma unroll
        for (int y = 0; y < EU / 4; ++y)
          rd[x][y] = raw4<IO_F32>(ab, (uint64_t)(uint32_t)(j < n ? j : n - 1) * (uint32_t)(b.heads * DK) + c + 4 * y);
      } else {
        rq[x] = *reinterpret_cast<const u32x4*>(qb + at_node(j, b.q_stride) + c);
      }
    }
  }
  typename Raw<IO>::Four wq[DIAG ? T::ROUNDS : 1][DK / 64];
  if constexpr (DIAG) {
#pragma unroll
    for (int t = 0; t < T::ROUNDS; ++t)
#pragma unroll
      for (int c = 0; c < DK / 64; ++c) wq[t][c] = raw4<IO>(qb, at_node(4 * (NW * t + wave) + g, b.q_stride) + 64 * c + 4 * lc);
  }
  float ra = 1.f, rbeta = 0.f;
  if (wave == 0) {
    if constexpr (!DIAG) ra = ab[(lane < n ? lane : n - 1) * b.heads];
    rbeta = b.beta[(t0 + (lane < n ? lane : n - 1)) * b.heads + h];
  }
  typename Raw<IO>::One rv[T::STAGED ? 1 : NT][4];           // this lane's, or units of all columns
  u32x4 rvu[T::STAGED ? T::VUNITS : 1];
  const int col0 = rb * T::C;                    // the workgroup's first value column
  auto v_in = [&](int x) { return (x + 1) * 64 * NW <= N * (T::C / 8) || x * 64 * NW + tid < N * (T::C / 8); };
  if constexpr (T::STAGED) {
#pragma unroll
    for (int x = 0; x < T::VUNITS; ++x) {
      const int u = x * 64 * NW + tid, j = u / (T::C / 8), c = col0 + u % (T::C / 8) * 8;
      if (!v_in(x)) continue;
      const auto* from = vb + at_node(j, b.v_stride);
      if (a.wide) {
        rvu[x] = *reinterpret_cast<const u32x4*>(from + (c < b.dv ? c : 0));
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y)
          rvu[x][y] = from[min(c + 2 * y, b.dv - 1)] | (uint32_t)from[min(c + 2 * y + 1, b.dv - 1)] << 16;
      }
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) rv[t][r] = vb[at_node(16 * t + 4 * g + r, b.v_stride) + rowc];
  }
  f32x4 s[KS][2];
  if (b.fresh && b.fresh[i]) {
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) s[kk][0] = s[kk][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    const float* S = b.S + (((int64_t)slot * b.heads + h) * b.dv + rowc) * DK + 4 * g;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        s[kk][y] = a.nt ? load_state<true>(S + 32 * kk + 16 * y) : load_state<false>(S + 32 * kk + 16 * y);
  }

  // ---- paths and decays.  A tree with a parent that is no earlier node is worked
  // as if it had none, so that no load waits for this one, and its outputs are NaN.
  const bool refused = __any(parent < -1 || parent >= lane);
  if (refused) parent = -1;
  if (wave == 0) {
    double l = DIAG ? 0.0 : log2_of(fabsf(ra));
    uint64_t mask = path_mask<!DIAG>(parent, lane, l);
    if (lane >= n) mask = 0;
    if constexpr (!DIAG) {
      const uint64_t neg = __ballot(lane < n && ra < 0.f);
      const float hi = (float)l;
      nl.hi[lane] = hi;
      nl.lo[lane] = (float)(l - (double)hi);
      nl.g[lane] = exp2_of(l) * (__popcll(neg & mask) & 1 ? -1.f : 1.f);
      if (lane == 0) nl.neg = neg;
    }
    nl.beta[lane] = lane < n ? rbeta : 0.f;
    nl.on[0][lane] = (uint32_t)mask;
    nl.on[1][lane] = (uint32_t)(mask >> 32);
    if (lane == 0) nl.spoilt = 0;
  }

  // Tile (tj, ti) of P or M, from the rows of q or k: a lane has row 16 tj + lc at
  // columns 16 ti + 4 g .. + 3.
  auto gram = [&](const __bf16* rows, int tj, int ti) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      bf16x8 x[NR], y[NR];
      get8<NR>(kl + (16 * ti + lc) * PK + 32 * kk + 8 * g, kRow, x);
      get8<NR>(rows + (16 * tj + lc) * PK + 32 * kk + 8 * g, kRow, y);
      d = mfma_parts<NO>(x, y, d);
    }
    const int j = 16 * tj + lc, i0 = 16 * ti + 4 * g;
    const float hj = nl.hi[j], lj = nl.lo[j];
    const f32x4 hi = *reinterpret_cast<const f32x4*>(&nl.hi[i0]), lo = *reinterpret_cast<const f32x4*>(&nl.lo[i0]);
    const uint32_t on = nl.on[ti >> 1][j] >> (i0 & 31);
    const uint64_t neg = nl.neg;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x = __builtin_amdgcn_exp2f((hj - hi[r]) + (lj - lo[r])) * d[r];
      if (neg) {
        const uint32_t n0 = (uint32_t)neg & (nl.on[0][j] ^ nl.on[0][i0 + r]);
        const uint32_t n1 = (uint32_t)(neg >> 32) & (nl.on[1][j] ^ nl.on[1][i0 + r]);
        x = (__popc(n0) + __popc(n1)) & 1 ? -x : x;
      }
      d[r] = on >> r & 1 ? x : 0.f;
    }
    return d;
  };
  // T of tile t from M's block there: column lc by forward substitution in every
  // lane group, which writes its four rows.  Rows behind the last node stay the
  // identity's; the second half is left out where it holds none.
  auto invert = [&](int t, const float* m, int pitch) {
    float x[16];
    uint32_t odd = 0;
    auto rows = [&](auto from) {
#pragma unroll
      for (int r = decltype(from)::value; r < decltype(from)::value + 8; ++r) {
        x[r] = lc == r ? 1.f : 0.f;
        float d = 0.f;
#pragma unroll
        for (int c = 0; c < r; c += 4) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(m + r * pitch + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < r) d = fmaf(y[e], x[c + e], d);
        }
        if (r > 0) x[r] = fmaf(-nl.beta[16 * t + r], d, x[r]);
        const bool fine = fabsf(x[r]) < kLargest;
        odd |= fine ? 0u : 1u << r;
        x[r] = fine ? x[r] : 0.f;
      }
    };
    rows(std::integral_constant<int, 0>());
    if (n > 16 * t + 8) {
      rows(std::integral_constant<int, 8>());
    } else {
#pragma unroll
      for (int r = 8; r < 16; ++r) x[r] = lc == r ? 1.f : 0.f;
    }
    if (__any(odd != 0)) {
#pragma unroll
      for (int o = 1; o < 16; o *= 2) odd |= __shfl_xor((int)odd, o);
      if (lane == 0) atomicOr(&nl.spoilt, (unsigned long long)odd << 16 * t);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float y = g == 0 ? x[r] : g == 1 ? x[4 + r] : g == 2 ? x[8 + r] : x[12 + r];
      __bf16* to = tl + (16 * t + 4 * g + r) * PT + lc;
#pragma unroll
      for (int p = 0; p < NO; ++p) {
        const __bf16 part = (__bf16)y;
        to[p * kT] = part;
        y -= (float)part;
      }
    }
  };
  // Four of a unit's elements as parts of a node row; as they are for the walk.
  auto four_of = [](u32x4 x, int y) {
    f32x4 z;
    if constexpr (IO == IO_F32) {
      z = __builtin_bit_cast(f32x4, x);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = widen<IO>((uint16_t)(x[2 * y + e / 2] >> 16 * (e & 1)));
    }
    return z;
  };
  auto put_unit = [&](__bf16* to, u32x4 x, int y) {
    if constexpr (IO == IO_BF16) *reinterpret_cast<u32x2*>(to) = u32x2{x[2 * y], x[2 * y + 1]};
    else put4<NR>(to, kRow, four_of(x, y));
  };
  auto put_v = [&] {
    if constexpr (T::STAGED) {
#pragma unroll
      for (int x = 0; x < T::VUNITS; ++x) {
        const int u = x * 64 * NW + tid, j = u / (T::C / 8);
        if (v_in(x)) *reinterpret_cast<u32x4*>(&vl[j * T::PC + u % (T::C / 8) * 8]) = rvu[x];
      }
    }
  };

  f32x4 done[DIAG ? 1 : T::TASKS];
  // Task x of the tiles of P and M that are kept as parts; false behind the last.
  auto task = [&](int x, int& tj, int& ti, bool& m) {
    m = x >= T::PTILES;
    if (m) {
      x -= T::PTILES;
      tj = x < 2 ? 1 : x < 4 ? 2 : 3;
      ti = x - (tj == 1 ? 0 : tj == 2 ? 2 : 4);
      return x < T::MTILES;
    }
    tj = x < 2 ? 0 : x < 4 ? 1 : x < 8 ? 2 : 3;
    ti = x - (tj == 0 ? 0 : tj == 1 ? 2 : tj == 2 ? 4 : 8);
    return true;
  };
  auto put_done = [&] {
    if constexpr (!DIAG) {
#pragma unroll
      for (int x = 0; x < T::TASKS; ++x) {
        int tj, ti;
        bool m;
        if (task(x * NW + NW - 1 - wave, tj, ti, m))
          put4<NO>((m ? mp : pp) + (16 * tj + lc) * PW + slot_order(16 * ti + 4 * g), kPart, done[x]);
      }
    }
  };

  if constexpr (!DIAG) {
    // ---- node rows to LDS as parts, then P, M and T
#pragma unroll
    for (int x = 0; x < T::UNITS; ++x) {
      const int u = x * 64 * NW + tid, j = u / ROWU, c = u % ROWU * EU;
      if (unit_in(x)) {
#pragma unroll
        for (int y = 0; y < EU / 4; ++y) {
          const int at = j * PK + slot_order(c + 4 * y);
          put_unit(kl + at, rk[x], y);
          put_unit(ql + at, rq[x], y);
        }
      }
    }
    if constexpr (!T::OVERLAY) put_v();
    __syncthreads();
    if constexpr (DELTA) {
      if (wave < NT) {
        const f32x4 d = gram(kl, wave, wave);
        float* m = ml + wave * 16 * PT;
        *reinterpret_cast<f32x4*>(m + lc * PT + 4 * g) = d;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        invert(wave, m, PT);
      }
    }
#pragma unroll
    for (int x = 0; x < T::TASKS; ++x) {
      int tj, ti;
      bool m;
      done[x] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (task(x * NW + NW - 1 - wave, tj, ti, m) && (m ? ti < tj : ti <= tj)) done[x] = gram(m ? kl : ql, tj, ti);
    }
    if constexpr (!T::OVERLAY) put_done();
  } else {
    // ---- rows of k and decays to LDS in fp32.  Sixteen lanes walk up from a node:
    // what is left of q (and alpha k) on the way is multiplied by the decays passed,
    // and with the k's met makes P and M.
    constexpr int NJ = DK / 64, EPT = DK / 16, R = T::ROUNDS;
    float* const kw = reinterpret_cast<float*>(lds);
    float* const aw = kw + N * PR;
#pragma unroll
    for (int x = 0; x < T::UNITS; ++x) {
      const int u = x * 64 * NW + tid, j = u / ROWU, c = u % ROWU * EU;
      if (unit_in(x)) {
#pragma unroll
        for (int y = 0; y < EU / 4; ++y) {
          *reinterpret_cast<f32x4*>(kw + j * PR + c + 4 * y) = four_of(rk[x], y);
          *reinterpret_cast<float4*>(aw + j * PR + c + 4 * y) = rd[x][y];
        }
      }
    }
    if constexpr (!T::LATE) put_v();
    float q[R][EPT], k[DELTA ? R : 1][EPT];
    int at[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int j = 4 * (NW * t + wave) + g;
      at[t] = j < n ? j : -1;
#pragma unroll
      for (int c = 0; c < NJ; ++c) widen4<IO>(&q[t][4 * c], wq[t][c]);
      if (j < N)
        for (int c = 4 * lc; c < 16 * (j / 16 + 1); c += 64) {
          *reinterpret_cast<f32x4*>(&pl[j * PP + c]) = f32x4{0.f, 0.f, 0.f, 0.f};
          if constexpr (DELTA) *reinterpret_cast<f32x4*>(&ml[j * PP + c]) = f32x4{0.f, 0.f, 0.f, 0.f};
        }
    }
    __syncthreads();
    if constexpr (DELTA) {
#pragma unroll
      for (int t = 0; t < R; ++t)
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(kw + (at[t] < 0 ? 0 : at[t]) * PR + 64 * c + 4 * lc);
#pragma unroll
          for (int e = 0; e < 4; ++e) k[t][4 * c + e] = y[e];
        }
    }
    while (true) {
      bool more = false;
#pragma unroll
      for (int t = 0; t < R; ++t) {
        if (!__any(at[t] >= 0)) continue;
        const int j = 4 * (NW * t + wave) + g, here = at[t] < 0 ? 0 : at[t];
        const bool on = at[t] >= 0;
        const int up = __shfl(parent, here);
        float p = 0.f, m = 0.f;
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          const f32x4 kk = *reinterpret_cast<const f32x4*>(kw + here * PR + 64 * c + 4 * lc);
          const f32x4 aa = *reinterpret_cast<const f32x4*>(aw + here * PR + 64 * c + 4 * lc);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p = fmaf(q[t][4 * c + e], kk[e], p);
            q[t][4 * c + e] *= on ? aa[e] : 1.f;
            if constexpr (DELTA) {
              m = fmaf(k[t][4 * c + e], kk[e], m);
              k[t][4 * c + e] *= on ? aa[e] : 1.f;
            }
          }
        }
        p = row_sum<16>(p);
        if constexpr (DELTA) m = row_sum<16>(m);
        if (on && lc == 0) {
          pl[j * PP + here] = p;
          if constexpr (DELTA)
            if (here != j) ml[j * PP + here] = m;
        }
        at[t] = on ? up : -1;
        more = true;
      }
      if (!more) break;
    }
    __syncthreads();                             // the walks are done with kw and aw
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int j = 4 * (NW * t + wave) + g;
      if (j < N) {
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          const int to = j * PK + slot_order(64 * c + 4 * lc);
          put4<NR>(ql + to, kRow, f32x4{q[t][4 * c], q[t][4 * c + 1], q[t][4 * c + 2], q[t][4 * c + 3]});
          if constexpr (DELTA) put4<NR>(kl + to, kRow, f32x4{k[t][4 * c], k[t][4 * c + 1], k[t][4 * c + 2], k[t][4 * c + 3]});
        }
      }
    }
    __syncthreads();
    if constexpr (DELTA)
      if (wave < NT) invert(wave, ml + 16 * wave * PP + 16 * wave, PP);
  }

  // ---- S q and S k: q's with the lane's node 16 t + lc and value columns 4 g .. + 3,
  // as the outputs are stored, k's with column lc and nodes 4 g .. + 3, as w is an operand
  f32x4 xq[NT], xk[DELTA ? NT : 1];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    xq[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (DELTA) xk[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    bf16x4 lo[NO], hi[NO];
    split4<NO>(s[kk][0], lo);
    split4<NO>(s[kk][1], hi);
    bf16x8 sp8[NO];
#pragma unroll
    for (int y = 0; y < NO; ++y) sp8[y] = join(lo[y], hi[y]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int at = (16 * t + lc) * PK + 32 * kk + 8 * g;
      bf16x8 x[NR];
      get8<NR>(ql + at, kRow, x);
      xq[t] = mfma_parts<NO>(sp8, x, xq[t]);
      if constexpr (DELTA) {
        get8<NR>(kl + at, kRow, x);
        xk[t] = mfma_parts<NO>(x, sp8, xk[t]);
      }
    }
  }
  if constexpr (!DIAG) {
    if constexpr (T::OVERLAY) {
      __syncthreads();                           // the node rows are done with
      put_done();
      put_v();
    }
    __syncthreads();
  } else if constexpr (DELTA) {
    __syncthreads();
    if constexpr (T::LATE) {
      put_v();
      __syncthreads();
    }
  }
  if (!T::STAGED && row0 >= b.dv) return;

  // Four values of two tiles (u and u + 1) of a row of P or M as an operand; with
  // fp32 values the second tile counts as 0 where it is not asked for.
  auto operand = [&](const float* f, const __bf16* parts, int t, int u, bool second, bf16x8 (&out)[NO]) {
    if constexpr (!DIAG) {
      get8<NO>(parts + (16 * t + lc) * PW + 16 * u + 8 * g, kPart, out);
    } else {
      const float* p = f + (16 * t + lc) * PP + 16 * u + 4 * g;
      bf16x4 lo[NO], hi[NO];
      split4<NO>(*reinterpret_cast<const f32x4*>(p), lo);
      split4<NO>(second ? *reinterpret_cast<const f32x4*>(p + 16) : f32x4{0.f, 0.f, 0.f, 0.f}, hi);
#pragma unroll
      for (int y = 0; y < NO; ++y) out[y] = join(lo[y], hi[y]);
    }
  };

  // ---- w
  uint32_t bad[2] = {};                          // bit 16 (t % 2) + r of word t / 2: w of node 16 t + 4 g + r is not finite
  auto finite = [&](f32x4 x, int t) {
    uint32_t odd = 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool fine = fabsf(x[r]) < kLargest;
      odd |= fine ? 0u : 1u << r;
      x[r] = fine ? x[r] : 0.f;
    }
    bad[t / 2] |= odd << 16 * (t % 2);
    return x;
  };
  bf16x4 w[NT][NO];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const f32x4 beta = *reinterpret_cast<const f32x4*>(&nl.beta[16 * t + 4 * g]);
    f32x4 x;
    if constexpr (T::STAGED) {
      const bf16x4 v = read_column4(reinterpret_cast<const __bf16*>(vl) + (16 * t + 4 * g + lc / 4) * T::PC + 16 * wave + 4 * (lc & 3));
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = widen<IO>((uint16_t)(__builtin_bit_cast(uint64_t, v) >> 16 * r));
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = widen<IO>(rv[t][r]);
    }
    if constexpr (DELTA) {
      f32x4 y = xk[t];
      if constexpr (!DIAG) y *= *reinterpret_cast<const f32x4*>(&nl.g[16 * t + 4 * g]);
#pragma unroll
      for (int u = 0; u < t; u += 2) {
        bf16x8 m[NO], o[NO];
        operand(ml, mp, t, u, u + 1 < t, m);
#pragma unroll
        for (int p = 0; p < NO; ++p) o[p] = join(w[u][p], u + 1 < t ? w[u + 1 < NT ? u + 1 : u][p] : bf16x4{});
        y = mfma_parts<NO>(m, o, y);
      }
      x -= y;
    }
    x *= beta;
    split4<NO>(finite(x, t), w[t]);
    if constexpr (DELTA) {
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = NO - 1; p >= 0; --p) {
        const bf16x4 m = *reinterpret_cast<const bf16x4*>(tl + p * kT + (16 * t + lc) * PT + 4 * g);
#pragma unroll
        for (int o = NO - 1 - p; o >= 0; --o)
          y = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, m), __builtin_bit_cast(s16x4, w[t][o]), y, 0, 0, 0);
      }
      split4<NO>(finite(y, t), w[t]);            // T w may overflow where T and w do not
    }
  }

  // ---- o
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if constexpr (!DIAG) xq[t] *= nl.g[16 * t + lc];
#pragma unroll
    for (int u = 0; u <= t; u += 2) {
      bf16x8 p[NO], x[NO];
      operand(pl, pp, t, u, u + 1 <= t, p);
#pragma unroll
      for (int y = 0; y < NO; ++y) x[y] = join(w[u][y], u + 1 <= t ? w[u + 1 < NT ? u + 1 : u][y] : bf16x4{});
      xq[t] = mfma_parts<NO>(x, p, xq[t]);
    }
  }
  const unsigned long long rows = DELTA ? nl.spoilt : 0;
  if (refused || rows || __any((bad[0] | bad[1]) != 0)) {      // nodes behind one that is not finite
    uint32_t lo = bad[0] << 4 * g, hi = bad[1] << 4 * g;
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      lo |= __shfl_xor((int)lo, o);
      hi |= __shfl_xor((int)hi, o);
    }
    lo |= (uint32_t)rows;
    hi |= (uint32_t)(rows >> 32);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t l = __shfl((int)lo, 4 * g + r), h2 = __shfl((int)hi, 4 * g + r);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (refused || (l & nl.on[0][16 * t + lc]) != 0 || (h2 & nl.on[1][16 * t + lc]) != 0)
          xq[t][r] = __uint_as_float(0x7FC00000u);
    }
  }
  auto* const ob = static_cast<typename Raw<IO>::One*>(b.o) + t0 * b.o_stride + hv;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int j = 16 * t + lc, c = row0 + 4 * g;
    if constexpr (T::STAGED) {                   // in v's place: no other wave reads these columns
      *reinterpret_cast<u32x2*>(&vl[j * T::PC + 16 * wave + 4 * g]) = u32x2{pair16<IO>(xq[t][0], xq[t][1]), pair16<IO>(xq[t][2], xq[t][3])};
    } else if (j < n) {
      float* to = ob + (uint64_t)(uint32_t)j * (uint32_t)b.o_stride + c;
      if (a.wide) {
        if (c < b.dv) *reinterpret_cast<f32x4*>(to) = xq[t];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (c + r < b.dv) to[r] = xq[t][r];
      }
    }
  }
  if constexpr (T::STAGED) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < T::VUNITS; ++x) {
      const int u = x * 64 * NW + tid, j = u / (T::C / 8), c = u % (T::C / 8) * 8;
      if (!v_in(x) || j >= n || col0 + c >= b.dv) continue;
      auto* to = ob + (uint64_t)(uint32_t)j * (uint32_t)b.o_stride + col0 + c;
      const u32x4 y = *reinterpret_cast<const u32x4*>(&vl[j * T::PC + c]);
      if (a.wide) {
        *reinterpret_cast<u32x4*>(to) = y;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col0 + c + e < b.dv) to[e] = (uint16_t)(y[e / 2] >> 16 * (e & 1));
      }
    }
  }
}

// Bytes of LDS and the workgroups a CU holds of it, for up to MT tiles of nodes.
template <int IO, int DK, int DELTA, int DIAG, int MT, int NW>
struct TreeLds {
  template <int NT>
  using T = TreeTile<IO, DK, DELTA, DIAG, NT, NW>;
  static constexpr int BYTES = T<1>::max2(T<1>::max2(T<1>::BYTES, T<MT >= 2 ? 2 : 1>::BYTES),
                                          T<1>::max2(T<MT >= 3 ? 3 : 1>::BYTES, T<MT >= 4 ? 4 : 1>::BYTES));
  // Waves of a SIMD: as many workgroups as LDS holds, and no more than leave the
  // registers that a wave needs (256 trees of 8 nodes as above: six waves 108 us,
  // five, which is two workgroups, 124; at six, the wave that makes T spills three.
  // The caps of the other instances follow this one and are not measured).
  static constexpr int HELD = 160 * 1024 / (BYTES + (int)sizeof(TreeNodes)) * NW / 4;
  static constexpr int FEWER = IO == IO_BF16 ? 0 : 1;    // parts take registers too
  static constexpr int MOST = DK == 128 ? (MT == 1 ? 6 : 5) - FEWER : (MT == 1 ? 7 : 6) - FEWER;
  static constexpr int WAVES = MT == 4 && MOST > 4 ? (HELD < 4 ? HELD : 4) : HELD < MOST ? HELD : MOST;
  static_assert(HELD > 0, "one workgroup fits");
};

template <int IO, int DK, int DELTA, int DIAG, int MT, int NW>
__global__ __launch_bounds__(64 * NW, (TreeLds<IO, DK, DELTA, DIAG, MT, NW>::WAVES)) void tree_kernel(TreeArgs a, int row_blocks) {
  __shared__ __align__(16) char lds[TreeLds<IO, DK, DELTA, DIAG, MT, NW>::BYTES];
  __shared__ __align__(16) TreeNodes nl;
  const SlotArgs& b = a.s;
  // Blocks go to the eight XCDs in turn; where a tree's blocks divide by eight, an
  // XCD takes neighbouring heads, which share rows of q and k in its L2.
  const int blocks = b.heads * row_blocks;
  int i, part;
  if (blocks % 8 == 0) {
    const int own = blocks / 8, x = blockIdx.x / 8;
    i = x / own;
    part = (int)(blockIdx.x % 8) * own + x % own;
  } else {
    i = blockIdx.x / blocks;
    part = blockIdx.x % blocks;
  }
  const int h = part / row_blocks, rb = part % row_blocks;
  const Span sp = span_of(b, i);
  if (sp.t1 <= sp.t0) return;
  const int slot = b.slots ? __builtin_amdgcn_readfirstlane(b.slots[i]) : i;
  if (slot < 0) return;
  const int64_t nodes = sp.t1 - sp.t0;
  if (slot >= b.nslots || nodes > a.max_nodes) {
    const int c = threadIdx.x % (16 * NW), row = rb * 16 * NW + c;
    if (row < b.dv)
      for (int64_t t = sp.t0 + threadIdx.x / (16 * NW); t < sp.t1; t += 4)
        store1<IO>(b.o, t * b.o_stride + (int64_t)h * b.dv + row, __uint_as_float(0x7FC00000u));
    return;
  }
  const int n = (int)nodes;
  // The tiles are a constant of each branch: with a condition on each of them the
  // registers of the tiles are copied at every one.
  auto head = [&](auto t) { tree_head<IO, DK, DELTA, DIAG, decltype(t)::value, NW>(a, lds, nl, i, h, rb, slot, sp.t0, n); };
  if (MT == 1 || n <= 16) return head(std::integral_constant<int, 1>());
  if constexpr (MT >= 2) {
    if (MT == 2 || n <= 32) return head(std::integral_constant<int, 2>());
  }
  if constexpr (MT >= 4) {
    if (n <= 48) return head(std::integral_constant<int, 3>());
    head(std::integral_constant<int, 4>());
  }
}

}  // namespace dev

// Eight waves where there are more than 64 value columns, so that P, M and T are made
// once for up to 128; four otherwise.  (Four waves with 32 columns each, tried with
// operands of two parts, took the same for large batches and longer for small ones: 9
// trees of 1-37 nodes, 16 heads 64x80 in binary16 14 us instead of 12, 24 of 9-25, 16
// heads 128x128 in fp32 with a diagonal decay 17 instead of 16.)
template <int IO, int DK, int DELTA, int DIAG>
hipError_t launch_tree_instance(const TreeArgs& a, hipStream_t s) {
  auto launch = [&](auto kernel, int waves) {
    const int row_blocks = (a.s.dv + 16 * waves - 1) / (16 * waves);
    const int64_t blocks = (int64_t)a.s.seqs * a.s.heads * row_blocks;
    if (!fits_launch(blocks, 64 * waves)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(64 * waves), 0, s, a, row_blocks);
    return hipGetLastError();
  };
  auto tiles = [&](auto w) {
    constexpr int NW = decltype(w)::value;
    return a.max_nodes <= 16   ? launch(dev::tree_kernel<IO, DK, DELTA, DIAG, 1, NW>, NW)
           : a.max_nodes <= 32 ? launch(dev::tree_kernel<IO, DK, DELTA, DIAG, 2, NW>, NW)
                               : launch(dev::tree_kernel<IO, DK, DELTA, DIAG, 4, NW>, NW);
  };
  return a.s.dv > 64 ? tiles(std::integral_constant<int, 8>()) : tiles(std::integral_constant<int, 4>());
}

template <int IO>
hipError_t launch_tree_type(const TreeArgs& a, int dk, int delta, int diag, hipStream_t s) {
  auto rule = [&](auto d) {
    constexpr int DK = decltype(d)::value;
    if (delta) return diag ? launch_tree_instance<IO, DK, 1, 1>(a, s) : launch_tree_instance<IO, DK, 1, 0>(a, s);
    return diag ? launch_tree_instance<IO, DK, 0, 1>(a, s) : launch_tree_instance<IO, DK, 0, 0>(a, s);
  };
  return dk == 128 ? rule(std::integral_constant<int, 128>()) : rule(std::integral_constant<int, 64>());
}

}  // namespace lsq
