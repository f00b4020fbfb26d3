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
// Without replacement Q_i+1 is 1 - q(x_1) - ... - q(x_i).  How far a row's sum is from one
// (1e-7 for an fp32 softmax) counts there Q's inverse times, so below 1/16 it is the sum of
// q over the tokens not tried: one more pass over the row, by the entry's own workgroup.
// Sums and products are fp64: tokens are whole numbers, and a cumulative sum or
// a ratio next to its border decides which.
//
// Bound by dependent reads: the offsets, the trees, the tokens' probabilities, then a
// row for each sum, each behind the one before (a chain of five nodes, 65536 tokens: 12-13
// us; 64 trees of 6-16, 131072 tokens: 11-16 us for the first sums, 3-8 for each later
// launch, 5 for the draw).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lsq_slots.h"

namespace lsq {
namespace dev {

constexpr int kMaxRuns = kMaxVocab / kRun;       // of a row; a wave sums a run
constexpr double kLittle = 1.0 / 16;             // a smaller Q is summed
constexpr int kSumWaves = 4;                     // of sum_kernel (8: 35 us as below instead of 34, 16: 36)

// Four floats at any 4-byte address.
struct Four {
  float x[4];
};
__device__ __forceinline__ Four load4(const float* p) {
  Four f;
  __builtin_memcpy(&f, p, sizeof f);
  return f;
}

// x of the lane that a DPP control names, 0 where it names none or the row is
// masked out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, (uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0u, (uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive sums over the lanes.
__device__ __forceinline__ double scan(double x) {
  x += dpp<0x111, 0xF>(x);                       // row_shr 1, 2, 4, 8: within 16 lanes
  x += dpp<0x112, 0xF>(x);
  x += dpp<0x114, 0xF>(x);
  x += dpp<0x118, 0xF>(x);
  x += dpp<0x142, 0xA>(x);                       // row_bcast 15 into rows 1 and 3: within 32
  x += dpp<0x143, 0xC>(x);                       // row_bcast 31 into rows 2 and 3
  return x;
}

__device__ __forceinline__ double lane_of(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// What is left of a node's target row: max(p - c q, 0), p itself where q is null (no
// child was rejected: c = 0, and q may be anything), or p without the tokens that the
// lanes hold in gone (-1: none) where the drafts have no probabilities.
struct Residual {
  const float* p;
  const float* q;
  double cut;
  int gone;
  int vocab;

  __device__ __forceinline__ double of(float px, float qx) const {
    return fmax(q ? (double)px - cut * (double)fmaxf(qx, 0.f) : (double)px, 0.0);   // a NaN counts as nothing
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

  // This lane's share of run r: four elements of every 256.
  __device__ __forceinline__ double share(int r, int lane) const {
    const int e0 = r * kRun, e1 = min(vocab, e0 + kRun);
    const uint64_t any = any_in(e0, e1);
    double sum = 0.0;
    if (e0 + kRun <= vocab && !any) {            // no branch between the loads: all in flight
      Four a[kRun / 256], b[kRun / 256] = {};
#pragma unroll
      for (int y = 0; y < kRun / 256; ++y) {
        a[y] = load4(p + e0 + 256 * y + 4 * lane);
        if (q) b[y] = load4(q + e0 + 256 * y + 4 * lane);
      }
#pragma unroll
      for (int y = 0; y < kRun / 256; ++y)
        sum += (of(a[y].x[0], b[y].x[0]) + of(a[y].x[1], b[y].x[1])) + (of(a[y].x[2], b[y].x[2]) + of(a[y].x[3], b[y].x[3]));
      return sum;
    }
#pragma unroll
    for (int y = 0; y < kRun; y += 256) {        // nothing behind the row
      double x[4];
      four(e0 + y + 4 * lane, any, x);
      sum += (x[0] + x[1]) + (x[2] + x[3]);
    }
    return sum;
  }
};

// The first lane whose inclusive sum (from base on) passes the threshold; where
// rounding leaves none, the last with something in it.  before: the sum up to it.
__device__ __forceinline__ int first_past(double own, double base, double threshold, int lane, double* before) {
  const double up = base + scan(own);
  const uint64_t past = __ballot(up > threshold && own > 0.0), some = __ballot(own > 0.0);
  const int at = past ? __builtin_ctzll(past) : some ? 63 - __builtin_clzll(some) : -1;
  if (at >= 0) *before = lane_of(up - own, at);
  return at;
}

// The whole sum of a row's runs, by one wave.
__device__ __forceinline__ double total_of(const double* sums, int runs, int lane) {
  double total = 0.0;
  for (int r0 = 0; r0 < runs; r0 += 64) {
    const double up = total + scan(r0 + lane < runs ? sums[r0 + lane] : 0.0);
    total = lane_of(up, 63);
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
    const double up = sum + scan(own);
    const uint64_t over = __ballot(up > threshold && own > 0.0), some = __ballot(own > 0.0);
    if (over || some) {                          // the last run with something, until one passes
      const int at = over ? __builtin_ctzll(over) : 63 - __builtin_clzll(some);
      run = r0 + at;
      before = lane_of(up - own, at);
    }
    if (over) break;
    sum = lane_of(up, 63);
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

// An entry's walk between two launches.
struct Saved {
  int done;                                      // the launch it ended in, counted from 1; 0: not yet, -1: a refused
                                                 // entry, -2 - k: it stopped in launch k and is left to verify_kernel
  int node, len, parent[kMaxNodes], id[kMaxNodes], took[kMaxNodes], gone[kMaxNodes];
  float u[kMaxNodes], px[kMaxNodes], qx[kMaxNodes];
  double cut, rest;
  uint64_t kids;
};
static_assert(sizeof(Saved) <= kSaved && kSaved % 16 == 0, "what the workspace holds");

// The walk of one entry, the same in every wave that makes it.
struct Walk {
  const VerifyArgs& a;
  int lane;
  int64_t t0;
  int parent, id;                                // of the lane's node
  float u, px, qx;                               // its uniform number, its token's chances in the rows of its parent
  bool sound, testable;
  int node, len, took;                           // where it is; lane d holds the path's node d
  uint64_t kids;                                 // children still to be tested
  double total, rest;
  bool stale;                                    // total is of an earlier cut
  Residual left;

  __device__ __forceinline__ Walk(const VerifyArgs& args, int i, int l) : a(args), lane(l) {
    t0 = min(max((int64_t)a.cu[i], (int64_t)0), a.nodes);
  }

  __device__ __forceinline__ const float* draft_row() const { return a.draft + (t0 + node) * a.draft_stride; }

  __device__ __forceinline__ void at_row(int j, double cut) {
    node = j;
    left.p = a.target + (t0 + j) * a.target_stride;
    left.cut = cut;
    left.q = cut > 0.0 ? draft_row() : nullptr;
    left.vocab = a.vocab;
  }

  __device__ __forceinline__ void at_node(int j) {
    at_row(j, 0.0);
    left.gone = -1;
    total = rest = 1.0;
    stale = false;
    kids = __ballot(testable && parent == j);
  }

  __device__ __forceinline__ void begin(int i) {
    const int64_t t1 = min(max((int64_t)a.cu[i + 1], (int64_t)0), a.nodes);
    const int n = (int)min(t1 - t0, (int64_t)kMaxNodes + 1);
    parent = lane < n ? a.parents[t0 + lane] : -1;
    sound = n > 0 && n <= kMaxNodes && !__any(parent < -1 || parent >= lane);
    id = lane < n ? a.ids[t0 + lane] : -1;
    u = lane < n ? a.uniform[t0 + lane] : 0.f;
    // every test's numbers at once
    testable = sound && lane < n && parent >= 0 && id >= 0 && id < a.vocab;
    px = 0.f, qx = 1.f;
    if (testable) {
      px = a.target[(t0 + parent) * a.target_stride + id];
      if (a.draft) qx = fmaxf(a.draft[(t0 + parent) * a.draft_stride + id], 0.f);
    }
    len = 1, took = lane == 0 ? 0 : -1;
    at_node(0);
  }

  // Goes on from where another launch stopped for want of the sum `known`.
  __device__ __forceinline__ void resume(const Saved& s, double known) {
    sound = true;
    parent = s.parent[lane], id = s.id[lane];
    u = s.u[lane], px = s.px[lane], qx = s.qx[lane];
    testable = parent >= 0 && id >= 0;
    len = s.len, took = s.took[lane];
    at_row(s.node, s.cut);
    left.gone = s.gone[lane];
    total = known, rest = s.rest, stale = false;
    kids = s.kids;
  }

  __device__ __forceinline__ void save(Saved& s, int done) const {
    s.parent[lane] = testable ? parent : -1, s.id[lane] = id, s.took[lane] = took, s.gone[lane] = left.gone;
    s.u[lane] = u, s.px[lane] = px, s.qx[lane] = qx;
    if (lane == 0) {
      s.node = node, s.len = len;
      s.cut = left.cut, s.rest = rest;
      s.kids = kids;
      s.done = done;
    }
  }

  // Whether the next test needs Q as a sum.
  __device__ __forceinline__ bool wants_rest() const { return stale && a.draft && !a.replacement && rest < kLittle; }

  // The node's draft row without the children tested so far.
  __device__ __forceinline__ Residual untried() const {
    const bool tested = testable && parent == node && !(kids >> lane & 1);
    return Residual{draft_row(), nullptr, 0.0, tested ? id : -1, a.vocab};
  }

  // Tests children until none is left or the path is full; sum(x) gives the sum of
  // x where a test needs it, or a negative number: then it stops there and returns
  // false.  In the end `left` is what the next token is drawn from.
  template <typename Sum>
  __device__ __forceinline__ bool run(Sum sum) {
    while (kids && len < a.depth) {
      for (bool q = wants_rest(); stale; q = false) {   // Q before T
        const double x = sum(q ? untried() : left);
        if (x < 0.0) return false;
        (q ? rest : total) = x;
        stale = q;
      }
      const int j = __builtin_ctzll(kids);
      kids &= kids - 1;
      const int x = __builtin_amdgcn_readlane(id, j);
      const float pj = __shfl(px, j);
      const double qj = __shfl(qx, j), uj = __shfl(u, j);
      const double pl = __any(left.gone == x) ? 0.0 : left.of(pj, (float)qj);
      if (uj * total * qj < pl * rest) {
        took = lane == len ? j : took;
        ++len;
        at_node(j);
      } else if (a.draft) {
        if (rest > 0.0) left.cut += total / rest;
        left.q = draft_row();
        if (!a.replacement) rest = fmax(rest - qj, 0.0);
        stale = true;
      } else {
        total = fmax(total - pl, 0.0);
        left.gone = lane == j ? x : left.gone;
      }
    }
    return true;
  }

  __device__ __forceinline__ void put_path(int i) const {
    for (int d = lane; d < a.depth; d += 64) a.path[(int64_t)i * a.depth + d] = sound && d < len ? took : -1;
    if (lane == 0) a.lengths[i] = sound ? len : 0;
  }
};

// The workspace: the runs' sums [rounds][seqs][runs], then the walks [rounds][seqs].
__device__ __forceinline__ double* sums_of(const VerifyArgs& a, int k, int i, int runs) {
  return a.ws + ((int64_t)k * a.seqs + i) * runs;
}

__device__ __forceinline__ Saved* saved_of(const VerifyArgs& a, int k, int i, int runs) {
  return reinterpret_cast<Saved*>(reinterpret_cast<char*>(a.ws + ((int64_t)a.rounds * a.seqs * runs + 1) / 2 * 2) +
                                  ((int64_t)k * a.seqs + i) * kSaved);
}

// The k-th sum of every entry that needs one: a wave per run.  The first wave of
// each workgroup makes the entry's walk up to there, from where the launch before
// left it; the entry's first workgroup writes down where that is.
__global__ __launch_bounds__(64 * kSumWaves) void sum_kernel(VerifyArgs a, int k) {
  __shared__ double cut;
  __shared__ int node, gone[kMaxNodes];          // node -1: nothing to sum
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int runs = (a.vocab + kRun - 1) / kRun, groups = (runs + kSumWaves - 1) / kSumWaves;
  const int i = blockIdx.x / groups, group = blockIdx.x % groups, r = group * kSumWaves + wave;
  Walk w(a, i, lane);
  if (wave == 0) {
    Saved& now = *saved_of(a, k, i, runs);
    int done = 0;
    if (k == 0) {
      w.begin(i);
    } else {
      const Saved& before = *saved_of(a, k - 1, i, runs);
      done = before.done;
      w.resume(before, total_of(sums_of(a, k - 1, i, runs), runs, lane));
    }
    if (done) {
      if (group == 0 && lane == 0) now.done = done;
    } else {
      // the walk's last sum is the one that the next token is drawn from
      const bool whole = w.sound && w.run([](const Residual&) { return -1.0; });
      if (w.sound && !whole && w.wants_rest()) done = -2 - k;
      if (group == 0) {
        w.save(now, !w.sound ? -1 : whole ? k + 1 : done);
        if (whole || !w.sound) w.put_path(i);
        if (!w.sound && lane == 0) a.next[i] = -1;
      }
    }
    gone[lane] = w.left.gone;
    if (lane == 0) {
      node = done || !w.sound ? -1 : w.node;
      cut = w.left.cut;
    }
  }
  __syncthreads();
  if (node < 0 || r >= runs) return;
  w.at_row(node, cut);
  w.left.gone = gone[lane];
  const double x = scan(w.left.share(r, lane));
  if (lane == 63) sums_of(a, k, i, runs)[r] = x;
}

// What the launches above left to do: the token of each entry, by one wave, and
// before it the walks that need more sums, with the whole workgroup.
constexpr int kWaves = 16;                       // of verify_kernel

__global__ __launch_bounds__(64 * kWaves) void verify_kernel(VerifyArgs a) {
  __shared__ double sums[kMaxRuns], buf[kRun / 64];
  const int lane = threadIdx.x & 63, i = blockIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int runs = (a.vocab + kRun - 1) / kRun, last = a.rounds - 1;
  const int done = a.rounds ? saved_of(a, last, i, runs)->done : 0;
  if (done == -1 || (done > 0 && wave != 0)) return;
  const double* from = sums;
  auto sum_runs = [&](const Residual& left, int first, int step) __attribute__((always_inline)) {
    for (int r = first; r < runs; r += 2 * step) {
      const double x = left.share(r, lane), y = r + step < runs ? left.share(r + step, lane) : 0.0;
      const double sx = scan(x), sy = scan(y);
      if (lane == 63) {
        sums[r] = sx;
        if (r + step < runs) sums[r + step] = sy;
      }
    }
  };
  Walk w(a, i, lane);
  if (done > 0) {
    from = sums_of(a, done - 1, i, runs);
    w.resume(*saved_of(a, done - 1, i, runs), 0.0);
  } else {
    if (done < 0) {
      w.resume(*saved_of(a, -2 - done, i, runs), 0.0);
      w.stale = true;
    } else if (a.rounds) {
      w.resume(*saved_of(a, last, i, runs), total_of(sums_of(a, last, i, runs), runs, lane));
    } else {
      w.begin(i);
    }
    if (!w.sound) {
      if (wave == 0) w.put_path(i);
      if (threadIdx.x == 0) a.next[i] = -1;
      return;
    }
    auto sum_row = [&](const Residual& x) __attribute__((always_inline)) {
      __syncthreads();
      sum_runs(x, wave, kWaves);
      __syncthreads();
    };
    w.run([&](const Residual& x) __attribute__((always_inline)) {
      sum_row(x);
      return total_of(sums, runs, lane);
    });
    sum_row(w.left);
    if (wave != 0) return;
    w.put_path(i);
  }
  const double part = fmin(fmax((double)a.uniform_next[i], 0.0), 1.0);
  int token = draw(w.left, from, runs, part, buf, lane);
  if (token < 0) {                               // nothing left: the token comes from p itself
    w.left.q = nullptr;
    w.left.gone = -1;
    sum_runs(w.left, 0, 1);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    token = draw(w.left, sums, runs, part, buf, lane);
  }
  if (lane == 0) a.next[i] = token;
}

}  // namespace dev

// An entry's own workgroup reads 60-110 GB/s: rows of 512 KiB and less are best left
// to it (one chain of five nodes, 65540 tokens: 13.6 us per call without launches
// for sums, 17.2, 19.9 and 22.4 with one to three, of which the host takes 2.6 each).
// Larger ones are split over the chip, by a launch for each sum; one that no entry
// needs takes 2-4 us.  The host does not see the trees: a chain asks for one sum,
// trees of 11 nodes for up to four (64 of them, 131072 tokens: 63 us without, 57, 47,
// 33, 34 and 37 with one to five).  Without a draft's row there is one sum.  Many
// rejected siblings of one node are slow either way, a sum behind the other (64 stars
// of 64 nodes, 65540 tokens: 569 us without launches, 556 with five).
int verify_rounds(int32_t seqs, int64_t nodes, int32_t vocab, bool draft) {
  if ((draft ? 2 : 1) * (int64_t)vocab <= 1 << 17 || seqs == 0) return 0;
  const int64_t rounds = draft ? (nodes / seqs - 3) / 2 : 1;
  return rounds < 1 ? 1 : rounds > 4 ? 4 : (int)rounds;
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  constexpr int per = dev::kSumWaves * kRun;
  const int64_t blocks = (int64_t)a.seqs * ((a.vocab + per - 1) / per);
  if (!fits_launch(a.seqs, 64 * dev::kWaves) || (a.rounds && !fits_launch(blocks, 64 * dev::kSumWaves)))
    return hipErrorInvalidConfiguration;
  for (int k = 0; k < a.rounds; ++k) {
    hipLaunchKernelGGL(dev::sum_kernel, dim3((unsigned)blocks), dim3(64 * dev::kSumWaves), 0, s, a, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(dev::verify_kernel, dim3((unsigned)a.seqs), dim3(64 * dev::kWaves), 0, s, a);
  return hipGetLastError();
}

}  // namespace lsq
