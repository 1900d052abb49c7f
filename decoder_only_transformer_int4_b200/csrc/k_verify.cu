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
// Bound: HBM for large vocabularies (one row of p and one of q per sequence), launch latency for
// small ones.  A cluster of CTAs shares a sequence's row: each warp sums a contiguous run, the
// runs' sums are exchanged over distributed shared memory, and the one warp whose run holds the
// border walks it again (it is in L1 or L2 by then).
#include <cooperative_groups.h>
#include <math.h>
#include "ms_device.cuh"
#include "ms_launch.cuh"
#include "ms_paged.h"

namespace ms {

namespace {
constexpr int kVerThreads = 256, kVerWarps = kVerThreads / 32, kVerMaxCluster = 8;

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
}  // namespace

__global__ void __launch_bounds__(kVerThreads) verify_draft_kernel(VerifyArgs a, unsigned* status) {
  namespace cg = cooperative_groups;
  __shared__ int first_refused;
  __shared__ double sums[2][kVerWarps];   // this CTA's runs: of the wanted weights, of p
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int r0 = a.row_start[b];
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
    return;   // the whole cluster: none waits at its barrier
  }
  const bool refused = taken < n;
  const float* p = a.target + (long long)(r0 + b + taken) * a.ldt;
  const float* q = refused && a.draft ? a.draft + (long long)(r0 + taken) * a.ldd : nullptr;
  const int banned = refused && !a.draft ? a.tokens[r0 + taken] : -1;
  auto rest = [&](int v, float pv, float qv) -> double {
    if (!refused) return pv;
    if (!q) return v == banned ? 0.0 : (double)pv;
    return fmax((double)pv - (double)qv, 0.0);
  };

  // this warp's run of the row
  const int runs = C * kVerWarps, len = (a.V + runs - 1) / runs;
  const int run = rank * kVerWarps + warp;
  const int v0 = min((long long)a.V, (long long)run * len), v1 = min(a.V, v0 + len);
  double s = 0.0, sp = 0.0;
  constexpr int U = 8;
  int v = v0 + lane;
  for (; v + 32 * (U - 1) < v1; v += 32 * U) {
    float pv[U], qv[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      pv[k] = p[v + 32 * k];
      qv[k] = q ? q[v + 32 * k] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      s += rest(v + 32 * k, pv[k], qv[k]);
      sp += pv[k];
    }
  }
  for (; v < v1; v += 32) {
    const float pv = p[v];
    s += rest(v, pv, q ? q[v] : 0.f);
    sp += pv;
  }
  s = warp_sum_d(s);
  sp = warp_sum_d(sp);
  if (lane == 0) {
    sums[0][warp] = s;
    sums[1][warp] = sp;
  }
  cluster.sync();
  // every warp reads all runs' sums (at most 64: two a lane) and finds the run with the border
  double x[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = 2 * lane + k;
    x[0][k] = x[1][k] = 0.0;
    if (r < runs) {
      const double* other = cluster.map_shared_rank(&sums[0][0], r / kVerWarps);
      x[0][k] = other[r % kVerWarps];
      x[1][k] = other[kVerWarps + r % kVerWarps];
    }
  }
  cluster.sync();   // no CTA leaves while another reads its sums
  const bool fall_back = !(warp_sum_d(x[0][0] + x[0][1]) > 0.0);
  const double a0 = fall_back ? x[1][0] : x[0][0], a1 = fall_back ? x[1][1] : x[0][1];
  double incl = a0 + a1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double z = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += z;
  }
  const double total = __shfl_sync(0xffffffffu, incl, 31);
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
  const double goal = (double)a.u_sample[b] * total;
  double before0 = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) before0 = 0.0;
  const double mid = before0 + a0;
  // the last run that begins at or below the goal and has any weight
  int r = -1;
  double at = 0.0;
  if (a0 > 0.0 && before0 <= goal) {
    r = 2 * lane;
    at = before0;
  }
  if (a1 > 0.0 && mid <= goal) {
    r = 2 * lane + 1;
    at = mid;
  }
  const unsigned has = __ballot_sync(0xffffffffu, r >= 0);
  const int from = has ? 31 - __clz(has) : 0;
  r = __shfl_sync(0xffffffffu, r, from);
  at = __shfl_sync(0xffffffffu, at, from);
  if (r != run) return;
  // this warp holds the border: walk its run in order
  int found = -1, last = -1;
  for (int w0 = v0; w0 < v1 && found < 0; w0 += 32) {
    const int w = w0 + lane;
    double y = 0.0;
    if (w < v1) y = fall_back ? (double)p[w] : rest(w, p[w], q ? q[w] : 0.f);
    double c = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double z = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) c += z;
    }
    const unsigned over = __ballot_sync(0xffffffffu, y > 0.0 && at + c > goal);
    const unsigned some = __ballot_sync(0xffffffffu, y > 0.0);
    if (over) found = w0 + __ffs(over) - 1;
    if (some) last = w0 + 31 - __clz(some);
    at += __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) out[taken] = found >= 0 ? found : last;   // last: the goal fell behind the run by rounding
}

cudaError_t launch_verify_draft(const Launch& L, const VerifyArgs& a) {
  // a CTA for each 4096 tokens of the row, up to a portable cluster
  int C = 1;
  while (C < kVerMaxCluster && C * 4096 < a.V) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.batch * C);
  cfg.blockDim = dim3(kVerThreads);
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)C, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = L.pdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_draft_kernel, a, L.status);
  if (e == cudaSuccess) launch_counter().fetch_add(1, std::memory_order_relaxed);
  return e;
}

}  // namespace ms
