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
// Precision: every operand is a sum of bf16 parts and the products of parts
// i + j < N are added; N = 3 (fp32) for fp32 inputs, N = 2 for 16-bit ones, whose
// outputs are rounded to 8 or 11 bits and whose states are not written.
//
// What is not finite would reach other paths through the zeros of P, M and T.  A
// w that is not counts as 0, and the outputs behind its node in its column become
// NaN; a row of T that is not counts as 0 and spoils all columns so.
template <int IO, int DK, int DELTA, int DIAG, int NT, int NW>
struct TreeTile {
  static constexpr int IN = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3;   // parts of an input
  static constexpr int NO = IO == IO_F32 ? 3 : 2;                       // parts of what is computed
  static constexpr int NR = DIAG ? NO : IN;                             // parts of the node rows
  static constexpr int N = 16 * NT, W = NT == 1 ? 32 : N;               // nodes; columns of P and M as parts
  // Pitches in elements: node rows, P and M as parts and as fp32, T, rows of the walk.
  static constexpr int PK = DK + 16, PW = W + 16, PP = N + 4, PT = 20, PR = DK + 4;
  static constexpr int EU = IO == IO_F32 ? 4 : 8;                       // elements of a 16-byte unit
  static constexpr int UNITS = (N * DK / EU + 64 * NW - 1) / (64 * NW); // units of q (k) per thread
  // 16-bit rows of v come, and of o go, through LDS: value columns of all waves, whole
  // 128-byte lines instead of 32-byte pieces.
  static constexpr bool STAGED = IO != IO_F32;
  static constexpr int C = 16 * NW, PC = C + 8, VUNITS = (N * C / 8 + 64 * NW - 1) / (64 * NW);
  static constexpr int ROUNDS = (4 * NT + NW - 1) / NW;                 // nodes a lane group walks up from
  static constexpr int PTILES = NT == 1 ? 2 : NT == 2 ? 4 : 12;         // tiles of P, with the zeros of a pair
  static constexpr int MTILES = !DELTA || NT == 1 ? 0 : NT == 2 ? 2 : 8;   // of M behind the first row of tiles
  static constexpr int TASKS = (PTILES + MTILES + NW - 1) / NW;
  // P and M as parts take the place of the node rows once the products with S are done.
  static constexpr bool OVERLAY = NT > 1;
  static constexpr int ROWS = 2 * NR * N * PK * (DIAG && !DELTA ? 1 : 2);   // bytes
  static constexpr int PARTS = DIAG ? 0 : 2 * NO * N * PW * (MTILES ? 2 : 1);
  static constexpr int RAW = DIAG ? 8 * N * PR : 0;
  static constexpr int max2(int x, int y) { return x > y ? x : y; }
  static constexpr int SHARED = max2(max2(ROWS + (OVERLAY ? 0 : PARTS), PARTS), RAW);
  static constexpr int BLOCKS = DIAG ? 4 * N * PP : 64 * NT * PT;       // bytes of M's (and P's) fp32 values
};

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

template <int IO, int DK, int DELTA, int DIAG, int NT, int NW>
__global__ __launch_bounds__(64 * NW, 2) void tree_kernel(TreeArgs a, int row_blocks) {
  using T = TreeTile<IO, DK, DELTA, DIAG, NT, NW>;
  constexpr int N = T::N, PK = T::PK, PP = T::PP, PW = T::PW, PT = T::PT, PR = T::PR, KS = DK / 32, NO = T::NO, NR = T::NR;
  constexpr int kRow = N * PK, kPart = N * PW, kT = NT * 16 * PT;      // planes
  __shared__ __align__(16) char shared[T::SHARED];
  __shared__ __align__(16) float pl[DIAG ? N * PP : 4];                // P in fp32
  __shared__ __align__(16) float ml[DELTA ? T::BLOCKS / 4 : 4];        // M in fp32, or its diagonal blocks
  __shared__ __align__(16) __bf16 tl[DELTA ? NO * kT : 8];
  __shared__ __align__(16) float hil[64], lol[64], gl[64], bl[64];
  __shared__ __align__(16) uint32_t onl[2][64];                        // the paths, by 32 nodes
  __shared__ uint64_t negl;
  __shared__ __align__(16) uint16_t vl[T::STAGED ? N * T::PC : 8];
  __shared__ unsigned long long spoiltl;
  __bf16* const ql = reinterpret_cast<__bf16*>(shared);
  __bf16* const kl = ql + NR * kRow;
  __bf16* const pp = T::OVERLAY ? ql : kl + NR * kRow;                 // P, then M, as parts
  __bf16* const mp = pp + NO * kPart;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
  const int64_t t0 = sp.t0, nodes = sp.t1 - sp.t0;
  const int row0 = (rb * NW + wave) * 16, row = row0 + lc;   // the lane's value column
  const int rowc = row < b.dv ? row : b.dv - 1;
  const int64_t hv = (int64_t)h * b.dv, hk = (int64_t)(h / b.share) * DK;
  if (slot >= b.nslots || nodes > a.max_nodes) {
    if (row < b.dv)
      for (int64_t t = t0 + g; t < sp.t1; t += 4) store1<IO>(b.o, t * b.o_stride + hv + row, __uint_as_float(0x7FC00000u));
    return;
  }
  const int n = (int)nodes, tiles = (n + 15) / 16;
  // Element offset of node j's row; rows behind the last repeat it.
  auto at_node = [&](int j, int64_t stride) { return (uint64_t)(uint32_t)(j < n ? j : n - 1) * (uint32_t)stride; };
  auto behind = [](const void* p, int64_t e) { return static_cast<const typename Raw<IO>::One*>(p) + e; };
  const auto* const kb = behind(b.k, t0 * b.k_stride + hk);
  const auto* const qb = behind(b.q, t0 * b.q_stride + hk);
  const auto* const vb = behind(b.v, t0 * b.v_stride + hv);
  const float* const ab = b.alpha + (t0 * b.heads + h) * (DIAG ? DK : 1);

  // ---- loads: node rows first, as they are used first
  int parent = lane < n ? a.parents[t0 + lane] : -1;
  constexpr int EU = T::EU, ROWU = DK / EU;      // units of a row
  auto unit_in = [&](int x) { return x * 64 * NW / ROWU < 16 * tiles && (N * ROWU % (64 * NW) == 0 || x * 64 * NW + tid < N * ROWU); };
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
  typename Raw<IO>::One rv[NT][4];               // this lane's, or units of all columns
  u32x4 ru[T::STAGED ? T::VUNITS : 1];
  const bool staged = T::STAGED && a.wide;
  const int col0 = rb * T::C;                    // the workgroup's first value column
  if (staged) {
#pragma unroll
    for (int x = 0; x < (T::STAGED ? T::VUNITS : 0); ++x) {
      const int u = x * 64 * NW + tid, j = u / (T::C / 8), c = col0 + u % (T::C / 8) * 8;
      if (j < 16 * tiles)
        ru[x] = *reinterpret_cast<const u32x4*>(vb + at_node(j, b.v_stride) + (c < b.dv ? c : 0));
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t < tiles) {
#pragma unroll
        for (int r = 0; r < 4; ++r) rv[t][r] = vb[at_node(16 * t + 4 * g + r, b.v_stride) + rowc];
      }
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
      hil[lane] = hi;
      lol[lane] = (float)(l - (double)hi);
      gl[lane] = exp2_of(l) * (__popcll(neg & mask) & 1 ? -1.f : 1.f);
      if (lane == 0) negl = neg;
    }
    bl[lane] = lane < n ? rbeta : 0.f;
    onl[0][lane] = (uint32_t)mask;
    onl[1][lane] = (uint32_t)(mask >> 32);
    if (lane == 0) spoiltl = 0;
  }

  // A tile of S's products' decayed cousins: rows tj of P (or M) at columns ti.
  auto gram = [&](const __bf16* rows, int tj, int ti) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      bf16x8 x[NR], y[NR];
      get8<NR>(rows + (16 * tj + lc) * PK + 32 * kk + 8 * g, kRow, x);
      get8<NR>(kl + (16 * ti + lc) * PK + 32 * kk + 8 * g, kRow, y);
      d = mfma_parts<NO>(x, y, d);
    }
    const int col = 16 * ti + lc, j0 = 16 * tj + 4 * g;
    const float hc = hil[col], lo = lol[col];
    const f32x4 hj = *reinterpret_cast<const f32x4*>(&hil[j0]), lj = *reinterpret_cast<const f32x4*>(&lol[j0]);
    const u32x4 on = *reinterpret_cast<const u32x4*>(&onl[ti >> 1][j0]);
    const uint64_t neg = negl;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float x = __builtin_amdgcn_exp2f((hj[r] - hc) + (lj[r] - lo)) * d[r];
      if (neg) {
        const uint32_t n0 = (uint32_t)neg & (onl[0][j0 + r] ^ onl[0][col]);
        const uint32_t n1 = (uint32_t)(neg >> 32) & (onl[1][j0 + r] ^ onl[1][col]);
        x = (__popc(n0) + __popc(n1)) & 1 ? -x : x;
      }
      d[r] = on[r] >> (col & 31) & 1 ? x : 0.f;
    }
    return d;
  };
  // T of tile t from M's block there: column lc by forward substitution in every
  // lane group, which writes its four rows.
  auto invert = [&](int t, const float* m, int pitch) {
    float x[16];
    uint32_t odd = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      x[r] = lc == r ? 1.f : 0.f;
      if (16 * t + r < n && r > 0) {
        float d = 0.f;
#pragma unroll
        for (int c = 0; c < r; c += 4) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(m + r * pitch + c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < r) d = fmaf(y[e], x[c + e], d);
        }
        x[r] = fmaf(-bl[16 * t + r], d, x[r]);
        const bool fine = fabsf(x[r]) <= 0x1.fffffep127f;
        odd |= fine ? 0u : 1u << r;
        x[r] = fine ? x[r] : 0.f;
      }
    }
    if (__any(odd != 0)) {
#pragma unroll
      for (int o = 1; o < 16; o *= 2) odd |= __shfl_xor((int)odd, o);
      if (lane == 0) atomicOr(&spoiltl, (unsigned long long)odd << 16 * t);
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
    if (staged) {
#pragma unroll
      for (int x = 0; x < (T::STAGED ? T::VUNITS : 0); ++x) {
        const int u = x * 64 * NW + tid, j = u / (T::C / 8);
        if (j < 16 * tiles) *reinterpret_cast<u32x4*>(&vl[j * T::PC + u % (T::C / 8) * 8]) = ru[x];
      }
    }
  };

  f32x4 done[DIAG ? 1 : T::TASKS];
  // Task x of the tiles of P and M that are kept as parts; false behind the last.
  auto task = [&](int x, int& tj, int& ti, bool& m) {
    const int np = tiles == 1 ? 2 : tiles == 2 ? 4 : tiles == 3 ? 8 : 12, nm = !DELTA ? 0 : tiles == 1 ? 0 : tiles == 2 ? 2 : tiles == 3 ? 4 : 8;
    m = x >= np;
    if (m) {
      x -= np;
      tj = x < 2 ? 1 : x < 4 ? 2 : 3;
      ti = x - (tj == 1 ? 0 : tj == 2 ? 2 : 4);
      return x < nm;
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
        if (task(x * NW + NW - 1 - wave, tj, ti, m)) {
          __bf16* to = (m ? mp : pp) + (16 * tj + 4 * g) * PW + slot_order(16 * ti + lc);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float y = done[x][r];
#pragma unroll
            for (int p = 0; p < NO; ++p) {
              const __bf16 part = (__bf16)y;
              to[p * kPart + r * PW] = part;
              y -= (float)part;
            }
          }
        }
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
    put_v();
    __syncthreads();
    if constexpr (DELTA) {
      if (wave < tiles) {
        const f32x4 d = gram(kl, wave, wave);
        float* m = ml + wave * 16 * PT;
#pragma unroll
        for (int r = 0; r < 4; ++r) m[(4 * g + r) * PT + lc] = d[r];
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
    float* const kw = reinterpret_cast<float*>(shared);
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
    put_v();
    float q[R][EPT], k[DELTA ? R : 1][EPT];
    int at[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
      const int j = 4 * (NW * t + wave) + g;
      at[t] = j < n ? j : -1;
#pragma unroll
      for (int c = 0; c < NJ; ++c) widen4<IO>(&q[t][4 * c], wq[t][c]);
      if (j < 16 * tiles)
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
      if (j < 16 * tiles) {
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
      if (wave < tiles) invert(wave, ml + 16 * wave * PP + 16 * wave, PP);
  }

  // ---- S q and S k
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
    for (int t = 0; t < NT; ++t)
      if (t < tiles) {
        const int at = (16 * t + lc) * PK + 32 * kk + 8 * g;
        bf16x8 x[NR];
        get8<NR>(ql + at, kRow, x);
        xq[t] = mfma_parts<NO>(x, sp8, xq[t]);
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
    }
    __syncthreads();
  } else if constexpr (DELTA) {
    __syncthreads();
  }
  if (!staged && row0 >= b.dv) return;

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
  uint32_t bad = 0;                              // bit 4 t + r: node 16 t + 4 g + r
  bf16x4 w[NT][NO];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t < tiles) {
      const f32x4 beta = *reinterpret_cast<const f32x4*>(&bl[16 * t + 4 * g]);
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (staged) rv[t][r] = vl[(16 * t + 4 * g + r) * T::PC + 16 * wave + lc];
        x[r] = widen<IO>(rv[t][r]);
      }
      if constexpr (DELTA) {
        f32x4 y = xk[t];
        if constexpr (!DIAG) y *= *reinterpret_cast<const f32x4*>(&gl[16 * t + 4 * g]);
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
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool fine = fabsf(x[r]) <= 0x1.fffffep127f;
        bad |= fine ? 0u : 1u << (4 * t + r);
        x[r] = fine ? x[r] : 0.f;
      }
      split4<NO>(x, w[t]);
      if constexpr (DELTA) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = NO - 1; p >= 0; --p) {
          const bf16x4 m = *reinterpret_cast<const bf16x4*>(tl + p * kT + (16 * t + lc) * PT + 4 * g);
#pragma unroll
          for (int o = NO - 1 - p; o >= 0; --o)
            y = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, m), __builtin_bit_cast(s16x4, w[t][o]), y, 0, 0, 0);
        }
        split4<NO>(y, w[t]);
      }
    }

  // ---- o
  uint64_t spoilt = 0;                           // nodes of the column whose w is not finite
  if (__any(bad != 0)) {
#pragma unroll
    for (int t = 0; t < NT; ++t) spoilt |= (uint64_t)(bad >> 4 * t & 15) << (16 * t + 4 * g);
#pragma unroll
    for (int o = 16; o < 64; o *= 2) {
      const uint32_t lo = __shfl_xor((int)(uint32_t)spoilt, o), hi = __shfl_xor((int)(uint32_t)(spoilt >> 32), o);
      spoilt |= (uint64_t)hi << 32 | lo;
    }
  }
  if constexpr (DELTA) spoilt |= spoiltl;
  const bool nans = refused || __any(spoilt != 0);
  auto* const ob = static_cast<typename Raw<IO>::One*>(b.o) + t0 * b.o_stride + hv;
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t < tiles) {
      f32x4 o = xq[t];
      if constexpr (!DIAG) o *= *reinterpret_cast<const f32x4*>(&gl[16 * t + 4 * g]);
#pragma unroll
      for (int u = 0; u <= t; u += 2) {
        bf16x8 p[NO], x[NO];
        operand(pl, pp, t, u, u + 1 <= t, p);
#pragma unroll
        for (int y = 0; y < NO; ++y) x[y] = join(w[u][y], u + 1 <= t ? w[u + 1 < NT ? u + 1 : u][y] : bf16x4{});
        o = mfma_parts<NO>(p, x, o);
      }
      if (nans) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * t + 4 * g + r;
          const bool hit = refused || ((uint32_t)spoilt & onl[0][j]) != 0 || ((uint32_t)(spoilt >> 32) & onl[1][j]) != 0;
          o[r] = hit ? __uint_as_float(0x7FC00000u) : o[r];
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * t + 4 * g + r;
        if constexpr (T::STAGED)
          if (staged) {                          // in v's place: no other wave reads these columns
            vl[j * T::PC + 16 * wave + lc] = to16<IO>(o[r]);
            continue;
          }
        if (j < n && row < b.dv) store1<IO>(ob, (uint64_t)(uint32_t)j * (uint32_t)b.o_stride + row, o[r]);
      }
    }
  if (staged) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < (T::STAGED ? T::VUNITS : 0); ++x) {
      const int u = x * 64 * NW + tid, j = u / (T::C / 8), c = u % (T::C / 8) * 8;
      if (j < n && col0 + c < b.dv)
        *reinterpret_cast<u32x4*>(ob + (uint64_t)(uint32_t)j * (uint32_t)b.o_stride + col0 + c) =
            *reinterpret_cast<const u32x4*>(&vl[j * T::PC + c]);
    }
  }
}

}  // namespace dev

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
