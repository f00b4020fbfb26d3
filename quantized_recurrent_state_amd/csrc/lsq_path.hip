// Accepted paths of drafted tokens written into the slots of an fp32 handle.
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
// outputs, the next token's vectors in flight.  Bound by the state's bytes, read
// and written once (256 slots of 32 heads 128x128 in fp32 with a diagonal decay, one to
// eight tokens each: 193 us, 5.9 TB/s; 64 slots in bf16 with the delta rule, 40% of
// them fresh: 43 us, 5.0).  Two tokens ahead are 199 and 42 us there, R = 2 211 and
// 43, R = 8 187 and 43.
template <int IO, int DK, int DELTA, int DIAG, int R, bool NT>
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
  Node<IO, DK, DIAG, R> next;
  next.read(b, token(0), h, row0, lr, lc);
  for (int t = 0; t < p.len; ++t) {
    const Node<IO, DK, DIAG, R> x = next;
    next.read(b, token(t + 1), h, row0, lr, lc);
    x.template advance<DELTA>(s);
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
hipError_t launch_path_instance(const PathArgs& a, hipStream_t s) {
  const int row_blocks = (a.s.dv + 16 * kRows - 1) / (16 * kRows);
  const int64_t blocks = (int64_t)a.s.seqs * a.s.heads * row_blocks;
  if (!fits_launch(blocks, 256)) return hipErrorInvalidConfiguration;
  const auto kernel = a.nt ? dev::path_kernel<IO, DK, DELTA, DIAG, kRows, true>
                           : dev::path_kernel<IO, DK, DELTA, DIAG, kRows, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, row_blocks);
  return hipGetLastError();
}

template <int IO, int DK>
hipError_t launch_path_rule(const PathArgs& a, int delta, int diag, hipStream_t s) {
  if (delta) return diag ? launch_path_instance<IO, DK, 1, 1>(a, s) : launch_path_instance<IO, DK, 1, 0>(a, s);
  return diag ? launch_path_instance<IO, DK, 0, 1>(a, s) : launch_path_instance<IO, DK, 0, 0>(a, s);
}

}  // namespace

hipError_t launch_path(const PathArgs& a, int io, int dk, int delta, int diag, hipStream_t s) {
  if (io == IO_F32) return dk == 128 ? launch_path_rule<IO_F32, 128>(a, delta, diag, s) : launch_path_rule<IO_F32, 64>(a, delta, diag, s);
  if (io == IO_F16) return dk == 128 ? launch_path_rule<IO_F16, 128>(a, delta, diag, s) : launch_path_rule<IO_F16, 64>(a, delta, diag, s);
  return dk == 128 ? launch_path_rule<IO_BF16, 128>(a, delta, diag, s) : launch_path_rule<IO_BF16, 64>(a, delta, diag, s);
}

}  // namespace lsq
