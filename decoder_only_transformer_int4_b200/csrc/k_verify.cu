// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Draft i of a sequence (token x, drawn from q_i) stays while u_i q_i(x) < p_i(x).  At the first
// that does not, the next token is drawn from max(p_i - q_i, 0) (from p_i where that is zero
// everywhere, which only rounding brings about); when all n stay, from p_n.  Kept tokens and the
// next one are then distributed as if each had been drawn from the target.  The draw is the inverse of
// the cumulative sum: the lowest v whose sum exceeds u times the total.
//
// Every comparison and sum is in double: u q is then exact, and a sum over 10^5 values is off by
// ~1e-15 of the total, where fp32 sums would move the border between neighbouring tokens by more
// than many of their probabilities.
//
// Bound: latency.  One row of p and one of q per sequence is 2 to 25 MB at 32 to 64 sequences, 0.4 to 4 us
// of HBM; the chain row range -> token -> p(x), q(x) -> row -> border is about five dependent loads long.
// A cluster of CTAs shares a sequence's row.  Each warp sums a contiguous run; every CTA writes its runs'
// sums into all CTAs of the cluster, so that one cluster barrier is the only wait; the warp whose run
// holds the border then narrows it 32 times at a step (each lane sums a contiguous piece, it is in L1 or L2
// by then) instead of walking it.  Walked 32 values a step, the border cost more than all else: 18.6 us for
// 64 sequences of 32003 tokens and 26.9 us for 32 of 100003, against 7.4 us and 8.3 us (4.5 us for one sequence of
// 1393 tokens).  512 threads a CTA (with half the threads, or half the CTAs: 10% to 30% more) and 64 registers, two CTAs an
// SM: with fewer the loads of a round do not fit (40 registers: 9.4 and 10.1 us).
#include <cooperative_groups.h>
#include <math.h>
#include "ms_device.cuh"
#include "ms_launch.cuh"
#include "ms_paged.h"

namespace ms {

namespace {
constexpr int kVerThreads = 512, kVerWarps = kVerThreads / 32, kVerMaxCluster = 8;
constexpr int kVerRuns = kVerMaxCluster * kVerWarps, kPerLane = kVerRuns / 32;

// max(d, 0), but NaN where d is: a row that holds one has no sum
__device__ __forceinline__ double rest(double d) { return d <= 0.0 ? 0.0 : d; }
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_scan_d(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double z = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += z;
  }
  return v;
}
}  // namespace

__global__ void __launch_bounds__(kVerThreads, 2) verify_draft_kernel(VerifyArgs a, unsigned* status) {
  namespace cg = cooperative_groups;
  __shared__ int first_refused;
  __shared__ double sums[kVerRuns];   // of the runs of the whole cluster
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster.barrier_arrive();   // waited for before the first write into another CTA: all have begun then
  pdl_wait();
  pdl_trigger();
  const int r0 = a.row_start[b];
  const float u = a.u_sample[b];
  int n = a.row_start[b + 1] - r0;
  const bool ok = n >= 0 && n <= a.max_draft && r0 >= 0 && r0 + (long long)n <= a.rows;
  if (!ok) n = 0;   // flagged below; every CTA of the cluster takes the same way out
  if (tid == 0) first_refused = n;
  __syncthreads();
  if (tid < n) {
    const int x = a.tokens[r0 + tid];
    bool stays = false;
    if (x >= 0 && x < a.V) {
      const double p = a.target[(long long)(r0 + b + tid) * a.ldt + x];
      const double q = a.draft ? (double)a.draft[(long long)(r0 + tid) * a.ldd + x] : 1.0;
      stays = (double)a.u_accept[r0 + tid] * q < p;
    } else if (rank == 0) {
      flag_error(status, kErrToken);
    }
    if (!stays) atomicMin(&first_refused, tid);
  }
  __syncthreads();
  const int taken = first_refused;
  int* out = a.out + (long long)b * (a.max_draft + 1);
  if (!ok) {
    if (rank == 0) {
      if (tid == 0) {
        flag_error(status, kErrShape);
        a.accepted[b] = 0;
      }
      for (int j = tid; j <= a.max_draft; j += kVerThreads) out[j] = -1;
    }
    cluster.barrier_wait();
    return;   // the whole cluster: none waits at its second barrier
  }
  const bool refused = taken < n;
  const float* p = a.target + (long long)(r0 + b + taken) * a.ldt;
  const float* q = refused && a.draft ? a.draft + (long long)(r0 + taken) * a.ldd : nullptr;
  int banned = refused && !a.draft ? a.tokens[r0 + taken] : -1;

  // this warp's run of the row
  const int runs = C * kVerWarps, len = (a.V + runs - 1) / runs;
  const int run = rank * kVerWarps + warp;
  const int v0 = min((long long)a.V, (long long)run * len), v1 = min(a.V, v0 + len);
  constexpr int U = 8;
  double x[kPerLane], mine, incl, total;
  cluster.barrier_wait();
  while (true) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};   // apart, so that additions do not wait for one another
    if (q) {
      for (int v = v0 + lane; v < v1; v += 32 * U) {
        float pv[U], qv[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const bool in = v + 32 * k < v1;
          pv[k] = in ? p[v + 32 * k] : 0.f;
          qv[k] = in ? q[v + 32 * k] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) s[k & 3] += rest((double)pv[k] - (double)qv[k]);
      }
    } else {
      for (int v = v0 + lane; v < v1; v += 64 * U) {
        float pv[2 * U];
#pragma unroll
        for (int k = 0; k < 2 * U; ++k) pv[k] = v + 32 * k < v1 ? p[v + 32 * k] : 0.f;
#pragma unroll
        for (int k = 0; k < 2 * U; ++k) s[k & 3] += v + 32 * k == banned ? 0.f : pv[k];
      }
    }
    const double all = warp_sum_d((s[0] + s[1]) + (s[2] + s[3]));
    if (lane < C) cluster.map_shared_rank(sums, lane)[run] = all;
    cluster.sync();
    mine = 0.0;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int r = kPerLane * lane + k;
      x[k] = r < runs ? sums[r] : 0.0;
      mine += x[k];
    }
    incl = warp_scan_d(mine, lane);
    total = __shfl_sync(0xffffffffu, incl, 31);
    if (!(total <= 0.0) || !(q || banned >= 0)) break;   // NaN is refused below
    q = nullptr;   // the whole cluster: p itself
    banned = -1;
    cluster.sync();   // the sums have been read
  }
  if (rank == 0 && warp == 0) {
    for (int j = lane; j <= a.max_draft; j += 32)
      if (j != taken) out[j] = j < taken ? a.tokens[r0 + j] : -1;
    if (lane == 0) a.accepted[b] = taken;
  }
  if (!(total > 0.0) || isinf(total)) {
    if (rank == 0 && tid == 0) {
      out[taken] = -1;
      flag_error(status, kErrToken);
    }
    return;
  }
  if (!(u >= 0.f && u < 1.f)) {
    if (rank == 0 && tid == 0) {
      out[taken] = -1;
      flag_error(status, kErrToken);
    }
    return;
  }
  const double goal = (double)u * total;
  double at = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) at = 0.0;
  // the last run that begins at or below the goal and has any weight
  int r = -1;
  double begin = 0.0;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    if (x[k] > 0.0 && at <= goal) {
      r = kPerLane * lane + k;
      begin = at;
    }
    at += x[k];
  }
  const unsigned has = __ballot_sync(0xffffffffu, r >= 0);
  const int from = has ? 31 - __clz(has) : 0;
  r = __shfl_sync(0xffffffffu, r, from);
  at = __shfl_sync(0xffffffffu, begin, from);
  if (r != run) return;
  // This warp holds the border.  [lo, hi) is narrowed to the piece of the first lane whose sum passes the
  // goal (the last with any weight, if the goal fell behind the run by rounding) until it is one value.
  int lo = v0, hi = v1;
  while (true) {
    const int step = (hi - lo + 31) / 32;
    const int w0 = min((long long)hi, lo + (long long)lane * step), w1 = min(hi, w0 + step);
    double part[2] = {0.0, 0.0};
    constexpr int N = 4;   // little code: one warp runs it, once, and waits for every line of it
    for (int w = w0; w < w1; w += N) {
      float pv[N], qv[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        pv[k] = w + k < w1 ? p[w + k] : 0.f;
        qv[k] = q && w + k < w1 ? q[w + k] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < N; ++k) part[k & 1] += w + k == banned ? 0.0 : rest((double)pv[k] - (double)qv[k]);
    }
    const double y = part[0] + part[1], c = at + warp_scan_d(y, lane);
    const unsigned over = __ballot_sync(0xffffffffu, y > 0.0 && c > goal);
    const unsigned some = __ballot_sync(0xffffffffu, y > 0.0);
    const int pick = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
    at = __shfl_sync(0xffffffffu, c - y, pick);
    lo = __shfl_sync(0xffffffffu, w0, pick);
    hi = __shfl_sync(0xffffffffu, w1, pick);
    if (step == 1) break;
  }
  if (lane == 0) out[taken] = lo;
}

cudaError_t launch_verify_draft(const Launch& L, const VerifyArgs& a, int n_sm) {
  // a CTA for each 8192 tokens of the row (16 a thread: one or two rounds of loads), up to a portable cluster and to two an
  // SM in all (43 sequences of 72091: 13.1 us in clusters of 4, 15.2 in more than fit at once)
  int C = 1;
  while (C < kVerMaxCluster && C * 8192 < a.V && (long long)a.batch * C * 2 <= 2 * n_sm) C *= 2;
  return launch_cluster(L, verify_draft_kernel, C, dim3(a.batch * C), dim3(kVerThreads), 0, a, L.status);
}

}  // namespace ms
