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
// mask, from the lanes' parents (-1 above a root): by pointer doubling, six
// rounds for any tree of 64 nodes.
__device__ __forceinline__ uint64_t path_mask(int parent, int lane) {
  uint64_t mask = (uint64_t)1 << lane;
  int up = parent;
#pragma unroll
  for (int r = 0; r < 6; ++r) {
    const int at = up < 0 ? lane : up;
    const uint32_t lo = __shfl((int)(uint32_t)mask, at), hi = __shfl((int)(uint32_t)(mask >> 32), at);
    const int next = __shfl(up, at);
    mask |= (uint64_t)hi << 32 | lo;
    if (up >= 0) up = next;
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
//   w         by forward substitution, 16 nodes at a time: earlier tiles by
//             products with M, the tile itself four nodes after four;
//   o         P w on top of g S q.
// A wave has 16 value columns from the state to the output; P and M are made
// once per workgroup.  Under a scalar decay D is 2^(L_j - L_i), L the sums of log2
// of the decays along the paths (fp64, held as two floats), with the sign of
// the negative ones between; under a diagonal one P and M are summed on the way up
// from each node, which leaves g_j k_j and g_j q_j for the products with S.
//
// Precision: every operand is a sum of bf16 parts and the products of parts
// i + j < N are added; N = 3 (fp32) for w and for fp32 outputs, N = 2 for the last
// products of 16-bit ones.  The substitution within a tile is fp32.
//
// A w that is not finite would reach other paths through P's and M's zeros.  It
// counts as 0, and the outputs behind its node in its column become NaN.
template <int IO, int DK, int DELTA, int DIAG, int NT>
struct TreeTile {
  static constexpr int IN = IO == IO_BF16 ? 1 : IO == IO_F16 ? 2 : 3;   // parts of an input
  static constexpr int NO = IO == IO_F32 ? 3 : 2;                       // parts on the output's side
  static constexpr int NQ = DIAG ? NO : IN, NK = DIAG ? 3 : IN;         // parts of the node rows
  static constexpr int NS = DELTA ? 3 : NO;                             // parts of the state
  static constexpr int N = 16 * NT, PK = DK + 16, PP = N + 4;           // nodes; pitches in elements
  static constexpr bool KROWS = !DIAG || DELTA;                         // rows of k are kept
  static constexpr int UNITS = N * DK / 4 / 256;                        // 4-element units of q (k) per thread
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

// Eight values of a row of P or M, four of each of two tiles, as N parts; the second
// four are 0 where that tile lies behind the row's.
template <int N>
__device__ __forceinline__ void operand(const float* p, bool second, bf16x8 (&out)[N]) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(p);
  const f32x4 hi = second ? *reinterpret_cast<const f32x4*>(p + 16) : f32x4{0.f, 0.f, 0.f, 0.f};
  bf16x4 a[N], b[N];
  split4<N>(lo, a);
  split4<N>(hi, b);
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = join(a[i], b[i]);
}

// Where element c of a row lies: the k-slots of lane group g hold elements
// 4 g .. 4 g + 3 of both halves of each 32, so that a 16-byte load of the state
// by every lane takes whole 64-byte runs of its rows.
__device__ __forceinline__ int slot_order(int c) { return (c & ~31) + 8 * ((c & 15) >> 2) + ((c & 16) >> 2) + (c & 3); }

// x as P parts to the rows' planes.
template <int P, typename Rows>
__device__ __forceinline__ void put4(Rows& dst, int at, f32x4 x) {
  bf16x4 p[P];
  split4<P>(x, p);
#pragma unroll
  for (int y = 0; y < P; ++y) *reinterpret_cast<bf16x4*>(&dst[y][at]) = p[y];
}

// Eight elements of a row's parts.
template <int P, typename Rows>
__device__ __forceinline__ void get8(const Rows& src, int at, bf16x8 (&out)[P]) {
#pragma unroll
  for (int y = 0; y < P; ++y) out[y] = *reinterpret_cast<const bf16x8*>(&src[y][at]);
}

template <int IO, int DK, int DELTA, int DIAG, int NT>
__global__ __launch_bounds__(256, 2) void tree_kernel(TreeArgs a, int row_blocks) {
  using T = TreeTile<IO, DK, DELTA, DIAG, NT>;
  constexpr int N = T::N, PK = T::PK, PP = T::PP, KS = DK / 32;
  __shared__ __align__(16) __bf16 ql[T::NQ][N * PK];
  __shared__ __align__(16) __bf16 kl[T::KROWS ? T::NK : 1][T::KROWS ? N * PK : 8];
  __shared__ __align__(16) float pl[N * PP];
  __shared__ __align__(16) float ml[DELTA ? N * PP : 4];
  __shared__ __align__(16) float hil[64], lol[64], gl[64], bl[64];
  __shared__ uint64_t maskl[64], negl;

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const SlotArgs& b = a.s;
  const int rb = blockIdx.x % row_blocks;
  const int64_t ih = blockIdx.x / row_blocks;
  const int h = (int)(ih % b.heads), i = (int)(ih / b.heads);
  const Span sp = span_of(b, i);
  if (sp.t1 <= sp.t0) return;
  const int slot = b.slots ? __builtin_amdgcn_readfirstlane(b.slots[i]) : i;
  if (slot < 0) return;
  const int64_t t0 = sp.t0, nodes = sp.t1 - sp.t0;
  const int row0 = rb * 64 + wave * 16, row = row0 + lc;     // the lane's value column
  const int rowc = row < b.dv ? row : b.dv - 1;
  const int64_t hv = (int64_t)h * b.dv, hk = (int64_t)(h / b.share) * DK;
  const int parent = lane < nodes ? a.parents[t0 + lane] : -1;
  if (slot >= b.nslots || nodes > a.max_nodes || __any(parent < -1 || parent >= lane)) {
    if (row < b.dv)
      for (int64_t t = t0 + g; t < sp.t1; t += 4) store1<IO>(b.o, t * b.o_stride + hv + row, __uint_as_float(0x7FC00000u));
    return;
  }
  const int n = (int)nodes, tiles = (n + 15) / 16;
  auto token = [&](int j) { return t0 + (j < n ? j : n - 1); };   // rows behind the last repeat it

  // ---- loads: node rows first, as they are used first
  typename Raw<IO>::Four rq[DIAG ? 1 : T::UNITS], rk[DIAG ? 1 : T::UNITS];
  if constexpr (!DIAG) {
#pragma unroll
    for (int x = 0; x < T::UNITS; ++x) {
      const int u = x * 256 + tid, j = u / (DK / 4), c = u % (DK / 4) * 4;
      if (x * 1024 / DK < 16 * tiles) {
        rk[x] = raw4<IO>(b.k, token(j) * b.k_stride + hk + c);
        rq[x] = raw4<IO>(b.q, token(j) * b.q_stride + hk + c);
      }
    }
  }
  float ra = 1.f, rbeta = 0.f;
  if (wave == 0) {
    if constexpr (!DIAG) ra = b.alpha[token(lane) * b.heads + h];
    rbeta = b.beta[token(lane) * b.heads + h];
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
  typename Raw<IO>::One rv[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t < tiles) {
#pragma unroll
      for (int r = 0; r < 4; ++r) rv[t][r] = raw1<IO>(b.v, token(16 * t + 4 * g + r) * b.v_stride + hv + rowc);
    }

  // ---- paths and decays
  if (wave == 0) {
    uint64_t mask = path_mask(parent, lane);
    if (lane >= n) mask = 0;
    if constexpr (!DIAG) {
      double l = log2_of(fabsf(ra));             // summed along the paths by pointer doubling
      int up = parent;
#pragma unroll
      for (int r = 0; r < 6; ++r) {
        const int at = up < 0 ? lane : up;
        const double add = __shfl(l, at);
        const int next = __shfl(up, at);
        if (up >= 0) {
          l += add;
          up = next;
        }
      }
      const uint64_t neg = __ballot(lane < n && ra < 0.f);
      const float hi = (float)l;
      hil[lane] = hi;
      lol[lane] = (float)(l - (double)hi);
      gl[lane] = exp2_of(l) * (__popcll(neg & mask) & 1 ? -1.f : 1.f);
      if (lane == 0) negl = neg;
    }
    bl[lane] = lane < n ? rbeta : 0.f;
    maskl[lane] = mask;
  }

  // ---- node rows to LDS as parts, P and M
  if constexpr (!DIAG) {
#pragma unroll
    for (int x = 0; x < T::UNITS; ++x) {
      const int u = x * 256 + tid, j = u / (DK / 4), c = u % (DK / 4) * 4;
      if (x * 1024 / DK < 16 * tiles) {
        const int at = j * PK + slot_order(c);
        float y[4];
        widen4<IO>(y, rk[x]);
        put4<T::NK>(kl, at, f32x4{y[0], y[1], y[2], y[3]});
        widen4<IO>(y, rq[x]);
        put4<T::NQ>(ql, at, f32x4{y[0], y[1], y[2], y[3]});
      }
    }
    __syncthreads();
    // tiles of the lower triangle, dealt over the waves
    const int pairs = tiles * (tiles + 1) / 2;
    const uint64_t neg = negl;
    auto decayed = [&](auto& rows, auto np, float* out, int at) {
      constexpr int P = decltype(np)::value, NA = sizeof(rows) / sizeof(rows[0]);
      const int tj = at >= 6 ? 3 : at >= 3 ? 2 : at >= 1 ? 1 : 0, ti = at - tj * (tj + 1) / 2;
      f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        bf16x8 x[NA], y[T::NK];
        get8<NA>(rows, (16 * tj + lc) * PK + 32 * kk + 8 * g, x);
        get8<T::NK>(kl, (16 * ti + lc) * PK + 32 * kk + 8 * g, y);
        d = mfma_parts<P>(x, y, d);
      }
      const int col = 16 * ti + lc;
      const float hc = hil[col], lo = lol[col];
      const uint64_t mc = maskl[col];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * tj + 4 * g + r;
        const uint64_t mj = maskl[j];
        float x = __builtin_amdgcn_exp2f((hil[j] - hc) + (lol[j] - lo)) * d[r];
        if (neg) x = __popcll(neg & mj & ~mc) & 1 ? -x : x;
        out[j * PP + col] = mj >> col & 1 ? x : 0.f;
      }
    };
    for (int x = wave; x < (DELTA ? 2 : 1) * pairs; x += 4) {
      if (x < pairs) decayed(ql, std::integral_constant<int, T::NO>(), pl, x);
      if constexpr (DELTA)
        if (x >= pairs) decayed(kl, std::integral_constant<int, 3>(), ml, x - pairs);
    }
  } else {
    // Sixteen lanes walk up from a node: what is left of q (and alpha k) on the way
    // is multiplied by the decays passed, and with the k's met makes P and M.
    constexpr int NJ = DK / 64, EPT = DK / 16;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t < tiles) {
        const int j = 16 * t + 4 * wave + g;
        for (int c = 4 * lc; c < 16 * (t + 1); c += 64) {
          *reinterpret_cast<f32x4*>(&pl[j * PP + c]) = f32x4{0.f, 0.f, 0.f, 0.f};
          if constexpr (DELTA) *reinterpret_cast<f32x4*>(&ml[j * PP + c]) = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        typename Raw<IO>::Four xq[NJ], xk[NJ];
        float4 xa[NJ];
        auto read = [&](int at) {
#pragma unroll
          for (int c = 0; c < NJ; ++c) {
            xk[c] = raw4<IO>(b.k, token(at) * b.k_stride + hk + 64 * c + 4 * lc);
            xa[c] = raw4<IO_F32>(b.alpha, (token(at) * b.heads + h) * DK + 64 * c + 4 * lc);
          }
        };
#pragma unroll
        for (int c = 0; c < NJ; ++c) xq[c] = raw4<IO>(b.q, token(j) * b.q_stride + hk + 64 * c + 4 * lc);
        read(j);
        float q[EPT], k[EPT];
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          widen4<IO>(&q[4 * c], xq[c]);
          widen4<IO>(&k[4 * c], xk[c]);
        }
        int at = j < n ? j : -1;
        while (__any(at >= 0)) {
          float kk[EPT], aa[EPT], p = 0.f, m = 0.f;
#pragma unroll
          for (int c = 0; c < NJ; ++c) {
            widen4<IO>(&kk[4 * c], xk[c]);
            widen4<IO_F32>(&aa[4 * c], xa[c]);
          }
          const bool on = at >= 0;
          const int here = at, up = __shfl(parent, on ? at : 0);
          at = on ? up : -1;
          read(at >= 0 ? at : 0);                // the next node's, in flight
#pragma unroll
          for (int e = 0; e < EPT; ++e) {
            p = fmaf(q[e], kk[e], p);
            if constexpr (DELTA) m = fmaf(k[e], kk[e], m);
            q[e] *= on ? aa[e] : 1.f;
            if constexpr (DELTA) k[e] *= on ? aa[e] : 1.f;
          }
          p = row_sum<16>(p);
          if constexpr (DELTA) m = row_sum<16>(m);
          if (on && lc == 0) {
            pl[j * PP + here] = p;
            if constexpr (DELTA)
              if (here != j) ml[j * PP + here] = m;
          }
        }
#pragma unroll
        for (int c = 0; c < NJ; ++c) {
          const int to = j * PK + slot_order(64 * c + 4 * lc);
          put4<T::NQ>(ql, to, f32x4{q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]});
          if constexpr (DELTA) put4<T::NK>(kl, to, f32x4{k[4 * c], k[4 * c + 1], k[4 * c + 2], k[4 * c + 3]});
        }
      }
    __syncthreads();
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
    bf16x4 lo[T::NS], hi[T::NS];
    split4<T::NS>(s[kk][0], lo);
    split4<T::NS>(s[kk][1], hi);
    bf16x8 sp8[T::NS];
#pragma unroll
    for (int y = 0; y < T::NS; ++y) sp8[y] = join(lo[y], hi[y]);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if (t < tiles) {
        const int at = (16 * t + lc) * PK + 32 * kk + 8 * g;
        bf16x8 x[T::NQ];
        get8<T::NQ>(ql, at, x);
        xq[t] = mfma_parts<T::NO>(x, sp8, xq[t]);
        if constexpr (DELTA) {
          bf16x8 y[T::NK];
          get8<T::NK>(kl, at, y);
          xk[t] = mfma_parts<3>(y, sp8, xk[t]);
        }
      }
  }
  if constexpr (!DIAG) __syncthreads();          // P and M are there
  if (row0 >= b.dv) return;

  // ---- w
  uint32_t bad = 0;                              // bit 4 t + r: node 16 t + 4 g + r
  auto finite = [&](float x, int bit, bool own) {
    const bool fine = fabsf(x) <= 0x1.fffffep127f;
    bad |= own && !fine ? 1u << bit : 0u;
    return fine ? x : 0.f;
  };
  bf16x4 w[NT][3];
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t < tiles) {
      const f32x4 beta = *reinterpret_cast<const f32x4*>(&bl[16 * t + 4 * g]);
      f32x4 x;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = widen<IO>(rv[t][r]);
      if constexpr (!DELTA) {
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = finite(beta[r] * x[r], 4 * t + r, true);
      } else {
        f32x4 y = xk[t];
        if constexpr (!DIAG) y *= *reinterpret_cast<const f32x4*>(&gl[16 * t + 4 * g]);
#pragma unroll
        for (int u = 0; u < t; u += 2) {
          bf16x8 m[3], o[3];
          operand<3>(&ml[(16 * t + lc) * PP + 16 * u + 4 * g], u + 1 < t, m);
#pragma unroll
          for (int p = 0; p < 3; ++p)
            o[p] = join(w[u][p], u + 1 < t ? w[u + 1 < NT ? u + 1 : u][p] : bf16x4{});
          y = mfma_parts<3>(m, o, y);
        }
        x -= y;
#pragma unroll
        for (int z = 0; z < 4; ++z) {            // the nodes of lane group z
          f32x4 m[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) m[r] = *reinterpret_cast<const f32x4*>(&ml[(16 * t + 4 * g + r) * PP + 16 * t + 4 * z]);
          f32x4 own, of;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float d = x[r];
#pragma unroll
            for (int c = 0; c < r; ++c) d = fmaf(-m[r][c], own[c], d);
            own[r] = finite(beta[r] * d, 4 * t + r, g == z);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) of[r] = __shfl(own[r], 16 * z + lc);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float d = x[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) d = fmaf(-m[r][c], of[c], d);
            x[r] = g == z ? own[r] : g > z ? d : x[r];
          }
        }
      }
      split4<3>(x, w[t]);
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
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t < tiles) {
      f32x4 o = xq[t];
      if constexpr (!DIAG) o *= *reinterpret_cast<const f32x4*>(&gl[16 * t + 4 * g]);
#pragma unroll
      for (int u = 0; u <= t; u += 2) {
        bf16x8 p[T::NO], x[T::NO];
        operand<T::NO>(&pl[(16 * t + lc) * PP + 16 * u + 4 * g], u + 1 <= t, p);
#pragma unroll
        for (int y = 0; y < T::NO; ++y) x[y] = join(w[u][y], u + 1 <= t ? w[u + 1 < NT ? u + 1 : u][y] : bf16x4{});
        o = mfma_parts<T::NO>(p, x, o);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * t + 4 * g + r;
        const float x = spoilt & maskl[j] ? __uint_as_float(0x7FC00000u) : o[r];
        if (j < n && row < b.dv) store1<IO>(b.o, (t0 + j) * b.o_stride + hv + row, x);
      }
    }
}

}  // namespace dev

template <int IO, int DK, int DELTA, int DIAG>
hipError_t launch_tree_instance(const TreeArgs& a, hipStream_t s) {
  const int row_blocks = (a.s.dv + 63) / 64;
  const int64_t blocks = (int64_t)a.s.seqs * a.s.heads * row_blocks;
  if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
  const auto kernel = a.max_nodes <= 16   ? dev::tree_kernel<IO, DK, DELTA, DIAG, 1>
                      : a.max_nodes <= 32 ? dev::tree_kernel<IO, DK, DELTA, DIAG, 2>
                                          : dev::tree_kernel<IO, DK, DELTA, DIAG, 4>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, row_blocks);
  return hipGetLastError();
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
