// Verification of drafted trees against the target's probabilities.
//
// At a node with target row p and draft row q the children x_1, x_2, ... are
// tested in order.  With P_1 = p, T_1 = Q_1 = 1, c_1 = 0, x_i is taken if
//   u T_i q(x_i) < P_i(x_i) Q_i;
// otherwise what is left is P_i+1 = max(P_i / T_i - q_i, 0) scaled by T_i, q_i = q / Q_i
// being the distribution x_i was drawn from.  Its positive part is that of
//   P_i+1 = max(p - c_i+1 q, 0),   c_i+1 = c_i + T_i / Q_i,
// (a rejected token has nothing left, P_i+1(x_i) = 0, so the q of a draw without
// replacement may keep the tokens drawn before), and T_i+1 is its sum.  One number c
// stands for all the rejections at a node, and a residual is never stored.
// Sums and products are fp64: tokens are whole numbers, and a cumulative sum or
// a ratio next to its border decides which.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"

namespace lsq {
namespace dev {

constexpr int kRun = 4096;                       // elements of a row that one wave sums
constexpr int kMaxRuns = kMaxVocab / kRun;       // of a row

// Four floats at any 4-byte address.
struct Four {
  float x[4];
};
__device__ __forceinline__ Four load4(const float* p) {
  Four f;
  __builtin_memcpy(&f, p, sizeof f);
  return f;
}

__device__ __forceinline__ double shfl_up(double x, int n) { return __shfl_up(x, n); }

// What is left of a node's target row: max(p - c q, 0), or p without the tokens
// that the lanes hold in gone (-1: none) where the drafts have no probabilities.
struct Residual {
  const float* p;
  const float* q;
  double cut;
  int gone;
  int vocab;

  __device__ __forceinline__ double of(float px, float qx) const {
    return fmax(q ? (double)px - cut * (double)qx : (double)px, 0.0);   // a NaN counts as nothing
  }

  // Four elements from e on, nothing behind the row; any: some token in gone
  // may be among the wave's.
  __device__ __forceinline__ void four(int e, uint64_t any, double (&x)[4]) const {
    Four a{}, b{};
    if (e + 4 <= vocab) {
      a = load4(p + e);
      if (q) b = load4(q + e);
    } else {
      for (int i = 0; i < 4; ++i)
        if (e + i < vocab) {
          a.x[i] = p[e + i];
          if (q) b.x[i] = q[e + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = of(a.x[i], b.x[i]);
    while (any) {
      const int t = __builtin_amdgcn_readlane(gone, __builtin_ctzll(any)) - e;
      any &= any - 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = t == i ? 0.0 : x[i];
    }
  }

  __device__ __forceinline__ uint64_t any_in(int e0, int e1) const { return __ballot(gone >= e0 && gone < e1); }

  // The sum of run r, in every lane.
  __device__ __forceinline__ double run(int r, int lane) const {
    const int e0 = r * kRun, e1 = min(vocab, e0 + kRun);
    const uint64_t any = any_in(e0, e1);
    double sum = 0.0;
#pragma unroll 4
    for (int e = e0 + 4 * lane; e < e1; e += 256) {
      double x[4];
      four(e, any, x);
      sum += (x[0] + x[1]) + (x[2] + x[3]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    return sum;
  }
};

// Inclusive sums over the lanes.
__device__ __forceinline__ double scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const double up = shfl_up(x, o);
    if (lane >= o) x += up;
  }
  return x;
}

// The first lane whose inclusive sum (from base on) passes the threshold; where
// rounding leaves none, the last with something in it.  before: the sum up to it.
__device__ __forceinline__ int first_past(double own, double base, double threshold, int lane, double* before) {
  const double up = base + scan(own, lane);
  const uint64_t past = __ballot(up > threshold && own > 0.0), some = __ballot(own > 0.0);
  const int at = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
  if (at >= 0) *before = __shfl(up - own, at);
  return at;
}

// The whole sum of a row's runs, by one wave, and with a threshold the run that
// passes it (the last with something in it where none does; -1 where nothing is left).
struct Found {
  double total, before;
  int run;
};

__device__ __forceinline__ Found over_runs(const double* sums, int runs, double threshold, int lane) {
  Found f{0.0, 0.0, -1};
  bool past = false;
  for (int r0 = 0; r0 < runs; r0 += 64) {
    const double own = r0 + lane < runs ? sums[r0 + lane] : 0.0;
    const double up = f.total + scan(own, lane);
    const uint64_t over = __ballot(up > threshold && own > 0.0), some = __ballot(own > 0.0);
    if (!past && (over || some)) {
      const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
      f.run = r0 + at;
      f.before = __shfl(up - own, at);
      past = over != 0;
    }
    f.total = __shfl(up, 63);
  }
  return f;
}

__global__ __launch_bounds__(1024) void verify_kernel(VerifyArgs a) {
  __shared__ double sums[kMaxRuns];
  const int lane = threadIdx.x & 63, i = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = min(max((int64_t)a.cu[i], (int64_t)0), a.nodes);
  const int64_t t1 = min(max((int64_t)a.cu[i + 1], (int64_t)0), a.nodes);
  const int n = (int)min(t1 - t0, (int64_t)kMaxNodes + 1);
  const int parent = lane < n ? a.parents[t0 + lane] : -1;
  const bool sound = n > 0 && n <= kMaxNodes && !__any(parent < -1 || parent >= lane);
  int* path = a.path + (int64_t)i * a.depth;
  if (!sound) {
    for (int d = threadIdx.x; d < a.depth; d += 1024) path[d] = -1;
    if (threadIdx.x == 0) {
      a.lengths[i] = 0;
      a.next[i] = -1;
    }
    return;
  }
  // Every test's numbers at once: node j's token, its probabilities in the rows
  // of its parent, its uniform number.
  const int id = lane < n ? a.ids[t0 + lane] : -1;
  const bool testable = lane < n && parent >= 0 && id >= 0 && id < a.vocab;
  double px = 0.0, qx = 1.0, u = 0.0;
  if (testable) {
    px = a.target[(t0 + parent) * a.target_stride + id];
    if (a.draft) qx = a.draft[(t0 + parent) * a.draft_stride + id];
    u = a.uniform[t0 + lane];
  }
  const int runs = (a.vocab + kRun - 1) / kRun;
  Residual left{nullptr, nullptr, 0.0, -1, a.vocab};
  auto at_node = [&](int j) {
    left.p = a.target + (t0 + j) * a.target_stride;
    left.q = a.draft ? a.draft + (t0 + j) * a.draft_stride : nullptr;
    left.cut = 0.0;
    left.gone = -1;
  };
  auto sum_runs = [&] {
    __syncthreads();
    for (int r = wave; r < runs; r += 16) {
      const double x = left.run(r, lane);
      if (lane == 0) sums[r] = x;
    }
    __syncthreads();
  };
  int cur = 0, len = 1, took = lane == 0 ? 0 : -1;         // took: lane d holds the path's node d
  double total = 1.0, rest = 1.0;
  bool stale = false, summed = false;            // total is of an earlier cut; sums are of this one
  at_node(0);
  uint64_t kids = __ballot(testable && parent == 0);
  while (kids && len < a.depth) {
    const int j = __builtin_ctzll(kids);
    kids &= kids - 1;
    const int x = __builtin_amdgcn_readlane(id, j);
    const double pj = __shfl(px, j), qj = __shfl(qx, j), uj = __shfl(u, j);
    if (stale) {
      sum_runs();
      total = over_runs(sums, runs, 0.0, lane).total;
      stale = false;
      summed = true;
    }
    const double pl = __any(left.gone == x) ? 0.0 : left.of((float)pj, (float)qj);
    if (uj * total * qj < pl * rest) {
      took = lane == len ? j : took;
      ++len;
      cur = j;
      at_node(j);
      total = rest = 1.0;
      summed = false;
      kids = __ballot(testable && parent == cur);
      continue;
    }
    summed = false;
    if (a.draft) {
      if (rest > 0.0) left.cut += total / rest;
      if (!a.replacement) rest = fmax(rest - qj, 0.0);
      stale = true;
    } else {
      total = fmax(total - pl, 0.0);
      left.gone = lane == j ? x : left.gone;
    }
  }
  if (!summed) sum_runs();
  double threshold = 0.0;
  const double un = fmin(fmax((double)a.uniform_next[i], 0.0), 1.0);
  Found f = over_runs(sums, runs, 0.0, lane);
  if (!(f.total > 0.0)) {                        // nothing left: the token comes from p itself
    left.q = nullptr;
    left.gone = -1;
    sum_runs();
    f = over_runs(sums, runs, 0.0, lane);
  }
  if (wave != 0) return;
  int token = -1;
  if (f.run >= 0) {
    threshold = un * f.total;
    f = over_runs(sums, runs, threshold, lane);
    const int e0 = f.run * kRun, e1 = min(a.vocab, e0 + kRun);
    const uint64_t any = left.any_in(e0, e1);
    double own = 0.0;                            // 64 elements in a row per lane
#pragma unroll 4
    for (int e = e0 + 64 * lane; e < min(e1, e0 + 64 * lane + 64); e += 4) {
      double x[4];
      left.four(e, any, x);
      own += (x[0] + x[1]) + (x[2] + x[3]);
    }
    double before = f.before;
    const int l = first_past(own, f.before, threshold, lane, &before);
    const int e = e0 + 64 * l + lane;            // then one per lane
    double x = e < e1 ? left.of(left.p[e], left.q ? left.q[e] : 0.f) : 0.0;
    for (uint64_t m = any; m; m &= m - 1)
      if (e == __builtin_amdgcn_readlane(left.gone, __builtin_ctzll(m))) x = 0.0;
    const int y = first_past(x, before, threshold, lane, &before);
    token = l < 0 || y < 0 ? -1 : e0 + 64 * l + y;
  }
  for (int d = lane; d < a.depth; d += 64) path[d] = d < len ? took : -1;
  if (lane == 0) {
    a.lengths[i] = len;
    a.next[i] = token;
  }
}

}  // namespace dev

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  if (!fits_launch(a.seqs, 1024)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(dev::verify_kernel, dim3((unsigned)a.seqs), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace lsq
