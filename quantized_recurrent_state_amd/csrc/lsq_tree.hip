// Drafted tokens over the slots of an fp32 handle: the recurrence along every
// path of a tree, and an accepted path written into the state.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"
#include "lsq_slots_dev.h"
#include "lsq_step_impl.h"

namespace lsq {
namespace dev {

// The rows of one wave, as in walk_kernel: sixteen lanes to a row, lane lc with
// columns 4 lc .. 4 lc + 3 of each 64, R rows a lane.
template <int IO, int DK, int DIAG, int R>
struct Node {
  static constexpr int NJ = DK / 64, EPT = DK / 16;
  typename Raw<IO>::Four k[NJ];
  float4 a[DIAG ? NJ : 1];
  typename Raw<IO>::One v[R];
  float alpha, beta;

  // Row t of the batch, of head h; rows behind dv repeat the last.
  __device__ __forceinline__ void read(const SlotArgs& b, int64_t t, int h, int row0, int lr, int lc) {
    const int64_t hk = (int64_t)(h / b.share) * DK;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      k[j] = raw4<IO>(b.k, t * b.k_stride + hk + 64 * j + 4 * lc);
      if constexpr (DIAG) a[j] = raw4<IO_F32>(b.alpha, (t * b.heads + h) * DK + 64 * j + 4 * lc);
    }
    if constexpr (!DIAG) alpha = b.alpha[t * b.heads + h];
    beta = b.beta[t * b.heads + h];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = row0 + 4 * r + lr;
      v[r] = raw1<IO>(b.v, t * b.v_stride + (int64_t)h * b.dv + (row < b.dv ? row : b.dv - 1));
    }
  }

  // One token of the recurrence, in walk_kernel's order of operations.
  template <int DELTA>
  __device__ __forceinline__ void advance(float (&s)[R][EPT]) const {
    float kk[EPT], aa[DIAG ? EPT : 1];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      widen4<IO>(&kk[4 * j], k[j]);
      if constexpr (DIAG) widen4<IO_F32>(&aa[4 * j], a[j]);
    }
    if constexpr (!DIAG) aa[0] = alpha;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float u = 0.f;
#pragma unroll
      for (int e = 0; e < EPT; ++e) s[r][e] *= aa[DIAG ? e : 0];
      if constexpr (DELTA) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) u = fmaf(s[r][e], kk[e], u);
        u = row_sum<16>(u);
      }
      const float w = beta * (widen<IO>(v[r]) - u);
#pragma unroll
      for (int e = 0; e < EPT; ++e) s[r][e] = fmaf(w, kk[e], s[r][e]);
    }
  }
};

template <int DK, int R, bool NT>
__device__ __forceinline__ void load_rows(float (&s)[R][DK / 16], const float* S, int row0, int dv, bool fresh,
                                          int lr, int lc) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 4 * r + lr;
#pragma unroll
    for (int j = 0; j < DK / 64; ++j) {
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
      if (!fresh && row < dv) x = load_state<NT>(S + (int64_t)row * DK + 64 * j + 4 * lc);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[r][4 * j + e] = x[e];
    }
  }
}

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

// Tree of one entry.  A wave holds its rows of the slot's state and walks every
// node's path from it.
template <int IO, int DK, int DELTA, int DIAG, int R>
__global__ __launch_bounds__(256) void tree_kernel(TreeArgs a, int row_blocks) {
  constexpr int NJ = DK / 64, EPT = DK / 16;
  const int lane = threadIdx.x & 63, lr = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const SlotArgs& b = a.s;
  const int rb = blockIdx.x % row_blocks;
  const int64_t ih = blockIdx.x / row_blocks;
  const int h = (int)(ih % b.heads), i = (int)(ih / b.heads);
  const int row0 = (rb * 4 + wave) * 4 * R;
  if (row0 >= b.dv) return;
  const Span sp = span_of(b, i);
  if (sp.t1 <= sp.t0) return;
  const int slot = b.slots ? __builtin_amdgcn_readfirstlane(b.slots[i]) : i;
  if (slot < 0) return;
  const int64_t n = sp.t1 - sp.t0;
  const int parent = lane < n ? a.parents[sp.t0 + lane] : -1;
  const int orow = row0 + 4 * lc + lr;          // the row whose output this lane stores
  const bool owrite = lc < R && orow < b.dv;
  if (slot >= b.nslots || n > a.max_nodes || __any(parent < -1 || parent >= lane)) {
    if (owrite)
      for (int64_t t = sp.t0; t < sp.t1; ++t)
        store1<IO>(b.o, t * b.o_stride + (int64_t)h * b.dv + orow, __uint_as_float(0x7FC00000u));
    return;
  }
  const uint64_t mask = path_mask(parent, lane);
  float s0[R][EPT];
  load_rows<DK, R, false>(s0, b.S + ((int64_t)slot * b.heads + h) * b.dv * DK, row0, b.dv,
                          b.fresh && b.fresh[i], lr, lc);
  for (int j = 0; j < n; ++j) {
    uint64_t on = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mask, j) |
                  (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(mask >> 32), j) << 32;
    float s[R][EPT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < EPT; ++e) s[r][e] = s0[r][e];
    while (on) {
      const int at = __builtin_ctzll(on);
      on &= on - 1;
      Node<IO, DK, DIAG, R> x;
      x.read(b, sp.t0 + at, h, row0, lr, lc);
      x.template advance<DELTA>(s);
    }
    float qq[EPT], out = 0.f;
#pragma unroll
    for (int c = 0; c < NJ; ++c)
      widen4<IO>(&qq[4 * c], raw4<IO>(b.q, (sp.t0 + j) * b.q_stride + (int64_t)(h / b.share) * DK + 64 * c + 4 * lc));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float o = 0.f;
#pragma unroll
      for (int e = 0; e < EPT; ++e) o = fmaf(s[r][e], qq[e], o);
      o = row_sum<16>(o);
      if (lc == r) out = o;
    }
    if (owrite) store1<IO>(b.o, (sp.t0 + j) * b.o_stride + (int64_t)h * b.dv + orow, out);
  }
}

// An entry's path: node numbers in the lanes, the slot it takes (kPadded for an
// entry with nothing to do).  One with a length of zero or less does nothing and takes no
// slot; one with more nodes than depth or a node outside its tree is refused.
struct Path {
  int64_t t0;
  int slot, len, node;
};

__device__ __forceinline__ Path path_of(const PathArgs& a, int i, int lane) {
  Path p{0, kPadded, 0, 0};
  const Span sp = span_of(a.s, i);
  p.t0 = sp.t0;
  p.len = __builtin_amdgcn_readfirstlane(a.lengths[i]);
  if (p.len <= 0) return p;
  p.slot = slot_of(a.s.slots, i, a.s.nslots, lane, [&](int j) { return a.lengths[j] > 0; });
  if (p.slot < 0) return p;
  if (p.len > a.depth) {
    p.slot = kRefused;
    return p;
  }
  p.node = lane < p.len ? a.path[(int64_t)i * a.depth + lane] : 0;
  if (__any(lane < p.len && (p.node < 0 || p.node >= sp.t1 - sp.t0))) p.slot = kRefused;
  return p;
}

// The accepted path: walk_kernel's token walk over the listed nodes, without
// outputs, the next D tokens' vectors in flight.
template <int IO, int DK, int DELTA, int DIAG, int R, int D, bool NT>
__global__ __launch_bounds__(256) void path_kernel(PathArgs a, int row_blocks) {
  constexpr int NJ = DK / 64, EPT = DK / 16;
  const int lane = threadIdx.x & 63, lr = lane >> 4, lc = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const SlotArgs& b = a.s;
  const int rb = blockIdx.x % row_blocks;
  const int64_t ih = blockIdx.x / row_blocks;
  const int h = (int)(ih % b.heads), i = (int)(ih / b.heads);
  const int row0 = (rb * 4 + wave) * 4 * R;
  if (row0 >= b.dv) return;
  const Path p = path_of(a, i, lane);
  if (p.slot < 0) return;
  float* S = b.S + ((int64_t)p.slot * b.heads + h) * b.dv * DK;
  float s[R][EPT];
  load_rows<DK, R, NT>(s, S, row0, b.dv, b.fresh && b.fresh[i], lr, lc);
  auto token = [&](int t) { return p.t0 + __builtin_amdgcn_readlane(p.node, t < p.len ? t : p.len - 1); };
  Node<IO, DK, DIAG, R> ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) ring[d].read(b, token(d), h, row0, lr, lc);
  for (int t = 0; t < p.len; t += D) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (t + d < p.len) {
        const Node<IO, DK, DIAG, R> x = ring[d];
        ring[d].read(b, token(t + d + D), h, row0, lr, lc);
        x.template advance<DELTA>(s);
      }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = row0 + 4 * r + lr;
    if (row < b.dv) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        store_state<NT>(S + (int64_t)row * DK + 64 * j + 4 * lc,
                        f32x4{s[r][4 * j], s[r][4 * j + 1], s[r][4 * j + 2], s[r][4 * j + 3]});
    }
  }
}

}  // namespace dev

namespace {

constexpr int kRows = 4;                         // rows a lane

template <int IO, int DK, int DELTA, int DIAG>
hipError_t launch_tree_instance(const TreeArgs& a, hipStream_t s) {
  const int row_blocks = (a.s.dv + 16 * kRows - 1) / (16 * kRows);
  const int64_t blocks = (int64_t)a.s.seqs * a.s.heads * row_blocks;
  if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((dev::tree_kernel<IO, DK, DELTA, DIAG, kRows>), dim3((unsigned)blocks), dim3(256), 0, s, a,
                     row_blocks);
  return hipGetLastError();
}

template <int IO, int DK, int DELTA, int DIAG>
hipError_t launch_path_instance(const PathArgs& a, hipStream_t s) {
  const int row_blocks = (a.s.dv + 16 * kRows - 1) / (16 * kRows);
  const int64_t blocks = (int64_t)a.s.seqs * a.s.heads * row_blocks;
  if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
  const auto kernel = a.nt ? dev::path_kernel<IO, DK, DELTA, DIAG, kRows, 1, true>
                           : dev::path_kernel<IO, DK, DELTA, DIAG, kRows, 1, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, row_blocks);
  return hipGetLastError();
}

// f.template operator()<IO, DK, DELTA, DIAG>() of the run-time choice.
template <int IO, int DK, typename F>
hipError_t by_rule(int delta, int diag, F f) {
  if (delta) return diag ? f.template operator()<IO, DK, 1, 1>() : f.template operator()<IO, DK, 1, 0>();
  return diag ? f.template operator()<IO, DK, 0, 1>() : f.template operator()<IO, DK, 0, 0>();
}

template <typename F>
hipError_t by_type(int io, int dk, int delta, int diag, F f) {
  if (io == IO_F32) return dk == 128 ? by_rule<IO_F32, 128>(delta, diag, f) : by_rule<IO_F32, 64>(delta, diag, f);
  if (io == IO_F16) return dk == 128 ? by_rule<IO_F16, 128>(delta, diag, f) : by_rule<IO_F16, 64>(delta, diag, f);
  return dk == 128 ? by_rule<IO_BF16, 128>(delta, diag, f) : by_rule<IO_BF16, 64>(delta, diag, f);
}

struct TreeLaunch {
  const TreeArgs& a;
  hipStream_t s;
  template <int IO, int DK, int DELTA, int DIAG>
  hipError_t operator()() const { return launch_tree_instance<IO, DK, DELTA, DIAG>(a, s); }
};

struct PathLaunch {
  const PathArgs& a;
  hipStream_t s;
  template <int IO, int DK, int DELTA, int DIAG>
  hipError_t operator()() const { return launch_path_instance<IO, DK, DELTA, DIAG>(a, s); }
};

}  // namespace

hipError_t launch_tree(const TreeArgs& a, int io, int dk, int delta, int diag, hipStream_t s) {
  return by_type(io, dk, delta, diag, TreeLaunch{a, s});
}

hipError_t launch_path(const PathArgs& a, int io, int dk, int delta, int diag, hipStream_t s) {
  return by_type(io, dk, delta, diag, PathLaunch{a, s});
}

}  // namespace lsq
