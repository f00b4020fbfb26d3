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

constexpr int kMaxRuns = kMaxVocab / kRun;       // of a row; a wave sums a run

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
    } else if (e < vocab) {
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

// The whole sum of a row's runs, by one wave.
__device__ __forceinline__ double total_of(const double* sums, int runs, int lane) {
  double total = 0.0;
  for (int r0 = 0; r0 < runs; r0 += 64) {
    const double up = total + scan(r0 + lane < runs ? sums[r0 + lane] : 0.0, lane);
    total = __shfl(up, 63);
  }
  return total;
}

// The first token whose cumulative sum passes `part` of the row's, by one wave,
// from the sums of its runs; -1 where nothing is left.  buf: kRun / 64 doubles of
// LDS for this wave.
__device__ __forceinline__ int draw(const Residual& left, const double* sums, int runs, double part, double* buf, int lane) {
  const double threshold = part * total_of(sums, runs, lane);
  int run = -1;
  double before = 0.0, sum = 0.0;
  for (int r0 = 0; r0 < runs; r0 += 64) {
    const double own = r0 + lane < runs ? sums[r0 + lane] : 0.0;
    const double up = sum + scan(own, lane);
    const uint64_t over = __ballot(up > threshold && own > 0.0), some = __ballot(own > 0.0);
    if (over || some) {                          // the last run with something, until one passes
      const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
      run = r0 + at;
      before = __shfl(up - own, at);
    }
    if (over) break;
    sum = __shfl(up, 63);
  }
  if (run < 0) return -1;
  constexpr int E = kRun / 64;                   // elements in a row per lane
  const int e0 = run * kRun, e1 = min(left.vocab, e0 + kRun), e = e0 + E * lane;
  const uint64_t any = left.any_in(e0, e1);
  double x[E], own = 0.0;
#pragma unroll
  for (int y = 0; y < E; y += 4) left.four(e + y, any, *reinterpret_cast<double (*)[4]>(&x[y]));
#pragma unroll
  for (int y = 0; y < E; y += 4) own += (x[y] + x[y + 1]) + (x[y + 2] + x[y + 3]);
  const int l = first_past(own, before, threshold, lane, &before);
  if (l < 0) return -1;
  if (lane == l) {                               // its elements, one per lane
#pragma unroll
    for (int y = 0; y < E; ++y) buf[y] = x[y];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int y = first_past(lane < E ? buf[lane] : 0.0, before, threshold, lane, &before);
  return y < 0 ? -1 : e0 + E * l + y;
}

// The walk of one entry, the same in every wave.  It asks for the sum of what is
// left of a row, in order, where a decision needs it: sum(k, left) of the k-th
// time returns it, or ends the walk with a negative number.
struct Walk {
  const VerifyArgs& a;
  int i, lane;
  int64_t t0;
  int n, parent, id;
  bool sound, testable;
  double px, qx, u;
  Residual left;
  int node, len, took;                           // the node it is at; lane d holds the path's node d

  __device__ __forceinline__ Walk(const VerifyArgs& args, int entry, int l) : a(args), i(entry), lane(l) {
    t0 = min(max((int64_t)a.cu[i], (int64_t)0), a.nodes);
    const int64_t t1 = min(max((int64_t)a.cu[i + 1], (int64_t)0), a.nodes);
    n = (int)min(t1 - t0, (int64_t)kMaxNodes + 1);
    parent = lane < n ? a.parents[t0 + lane] : -1;
    sound = n > 0 && n <= kMaxNodes && !__any(parent < -1 || parent >= lane);
    id = lane < n ? a.ids[t0 + lane] : -1;
    u = lane < n ? a.uniform[t0 + lane] : 0.f;
    at_node(0);
    len = 0, took = -1;
    // every test's numbers at once: a token's probabilities in the rows of its parent
    testable = sound && lane < n && parent >= 0 && id >= 0 && id < a.vocab;
    px = 0.0, qx = 1.0;
    if (testable) {
      px = a.target[(t0 + parent) * a.target_stride + id];
      if (a.draft) qx = a.draft[(t0 + parent) * a.draft_stride + id];
    }
  }

  __device__ __forceinline__ void at_node(int j) {
    node = j;
    left.p = a.target + (t0 + j) * a.target_stride;
    left.q = a.draft ? a.draft + (t0 + j) * a.draft_stride : nullptr;
    left.cut = 0.0;
    left.gone = -1;
    left.vocab = a.vocab;
  }

  // False where a sum was not to be had.  Ends with `left` at the last node.
  template <typename Sum>
  __device__ __forceinline__ bool run(Sum sum) {
    len = 1, took = lane == 0 ? 0 : -1;
    int sums = 0;                                // asked for so far
    double total = 1.0, rest = 1.0;
    bool stale = false;                          // total is of an earlier cut
    at_node(0);
    uint64_t kids = __ballot(testable && parent == 0);
    while (kids && len < a.depth) {
      const int j = __builtin_ctzll(kids);
      kids &= kids - 1;
      const int x = __builtin_amdgcn_readlane(id, j);
      const double pj = __shfl(px, j), qj = __shfl(qx, j), uj = __shfl(u, j);
      if (stale) {
        total = sum(sums++);
        if (total < 0.0) return false;
        stale = false;
      }
      const double pl = __any(left.gone == x) ? 0.0 : left.of((float)pj, (float)qj);
      if (uj * total * qj < pl * rest) {
        took = lane == len ? j : took;
        ++len;
        at_node(j);
        total = rest = 1.0;
        kids = __ballot(testable && parent == j);
      } else if (a.draft) {
        if (rest > 0.0) left.cut += total / rest;
        if (!a.replacement) rest = fmax(rest - qj, 0.0);
        stale = true;
      } else {
        total = fmax(total - pl, 0.0);
        left.gone = lane == j ? x : left.gone;
      }
    }
    return true;
  }
};

// Where an entry's walk ended, behind the sums in the workspace.
struct Ended {
  int done;                                      // the number of sums then made; 0: not yet, -1: a refused entry
  int node;
  double cut;
  int gone[kMaxNodes];
};
static_assert(sizeof(Ended) == kEnded, "what the workspace holds");

__device__ __forceinline__ Ended* ended_of(const VerifyArgs& a, int runs) {
  return reinterpret_cast<Ended*>(a.ws + (int64_t)a.seqs * a.rounds * runs);
}

// Outputs of an entry whose walk has ended, by one wave; of a refused one with len 0.
__device__ __forceinline__ void put_path(const VerifyArgs& a, int i, int len, int took, int lane) {
  for (int d = lane; d < a.depth; d += 64) a.path[(int64_t)i * a.depth + d] = d < len ? took : -1;
  if (lane == 0) a.lengths[i] = len;
}

// The k-th sum of every entry that needs one: a wave per run, the runs' sums to the
// workspace [entries][rounds][runs].  Each wave makes the entry's walk by itself,
// from the sums of the rounds before; the first tells where it ended.
__global__ __launch_bounds__(256) void sum_kernel(VerifyArgs a, int k) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int runs = (a.vocab + kRun - 1) / kRun, groups = (runs + 3) / 4;
  const int i = blockIdx.x / groups, r = blockIdx.x % groups * 4 + wave;
  if (r >= runs) return;
  Ended* const end = ended_of(a, runs) + i;
  if (k > 0) {                                   // ended before; k + 1 is this launch's own word
    const int done = end->done;
    if (done < 0 || (done > 0 && done <= k)) return;
  }
  Walk w(a, i, lane);
  double* const ws = a.ws + (int64_t)i * a.rounds * runs;
  // the walk's last sum is the one that the next token is drawn from
  const bool whole = w.sound && w.run([&](int m) { return m < k ? total_of(ws + (int64_t)m * runs, runs, lane) : -1.0; });
  if (w.sound) {
    const double x = w.left.run(r, lane);
    if (lane == 0) ws[(int64_t)k * runs + r] = x;
  }
  if (r != 0) return;
  if (whole || !w.sound) {
    put_path(a, i, w.sound ? w.len : 0, w.took, lane);
    end->gone[lane] = w.left.gone;
  }
  if (lane == 0) {
    if (!w.sound) a.next[i] = -1;
    end->node = w.node;
    end->cut = w.left.cut;
    end->done = !w.sound ? -1 : whole ? k + 1 : 0;
  }
}

__global__ __launch_bounds__(1024) void verify_kernel(VerifyArgs a) {
  __shared__ double sums[kMaxRuns], buf[kRun / 64];
  const int lane = threadIdx.x & 63, i = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int runs = (a.vocab + kRun - 1) / kRun;
  const double* const ws = a.ws + (int64_t)i * a.rounds * runs;
  const double part = fmin(fmax(a.uniform_next ? (double)a.uniform_next[i] : 0.0, 0.0), 1.0);
  const Ended* const end = ended_of(a, runs) + i;
  const int done = a.rounds ? end->done : 0;
  if (done < 0 || (done && wave != 0)) return;
  Residual left{nullptr, nullptr, 0.0, -1, a.vocab};
  const double* from = sums;
  auto sum_runs = [&](int w0, int step) {        // waves w0, w0 + step, ...
    for (int r = w0; r < runs; r += step) {
      const double x = left.run(r, lane);
      if (lane == 0) sums[r] = x;
    }
  };
  if (done) {                                    // one wave draws
    const int64_t row = min(max((int64_t)a.cu[i], (int64_t)0), a.nodes) + end->node;
    left.p = a.target + row * a.target_stride;
    left.q = a.draft ? a.draft + row * a.draft_stride : nullptr;
    left.cut = end->cut;
    left.gone = end->gone[lane];
    from = ws + (int64_t)(done - 1) * runs;
  } else {
    Walk w(a, i, lane);
    if (!w.sound) {
      if (wave != 0) return;
      put_path(a, i, 0, -1, lane);
      if (lane == 0) a.next[i] = -1;
      return;
    }
    auto sum_row = [&] {
      left = w.left;
      __syncthreads();
      sum_runs(wave, 16);
      __syncthreads();
    };
    w.run([&](int m) {
      if (m < a.rounds) return total_of(ws + (int64_t)m * runs, runs, lane);
      sum_row();
      return total_of(sums, runs, lane);
    });
    sum_row();                                   // of the last row: no launch made it
    if (wave != 0) return;
    put_path(a, i, w.len, w.took, lane);
  }
  int token = draw(left, from, runs, part, buf, lane);
  if (token < 0) {                               // nothing left: the token comes from p itself
    left.q = nullptr;
    left.gone = -1;
    sum_runs(0, 1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    token = draw(left, sums, runs, part, buf, lane);
  }
  if (lane == 0) a.next[i] = token;
}

}  // namespace dev

// A sum made by a launch of its own takes about 5 us and 2.6 of the host, an idle
// launch 1.2; the entry's own workgroup takes 10 us for rows of 131072 tokens, and
// 2 for 16384.  The host does not see the trees: a chain asks for one sum, trees of 11
// nodes for four to five where they ask most (64 of them, 131072 tokens: 72 us
// without such launches, 69, 65, 53, 50 and 52 with one to five; one chain of five
// nodes, 65536 tokens: 16.1, 16.1, 18.7, 21.3).
int verify_rounds(int32_t seqs, int64_t nodes, int32_t vocab, bool draft) {
  if (vocab <= 4 * kRun || seqs == 0) return 0;
  if (!draft || vocab < (1 << 15)) return 1;     // without a draft's row there is one sum
  const int64_t rounds = (nodes / seqs - 3) / 2;
  return rounds < 1 ? 1 : rounds > 4 ? 4 : (int)rounds;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  const int64_t blocks = (int64_t)a.seqs * ((a.vocab + 4 * kRun - 1) / (4 * kRun));
  if (!fits_launch(a.seqs, 1024) || (a.rounds && !fits_launch(blocks, 256))) return hipErrorInvalidConfiguration;
  for (int k = 0; k < a.rounds; ++k) {
    hipLaunchKernelGGL(dev::sum_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(dev::verify_kernel, dim3((unsigned)a.seqs), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace lsq
