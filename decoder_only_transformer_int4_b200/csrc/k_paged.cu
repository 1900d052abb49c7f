// Rotary positions with the append into a paged cache, and eviction from it by accumulated
// attention weight.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include "ms_device.cuh"
#include "ms_launch.cuh"
#include "ms_paged.h"

namespace ms {

namespace {

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T e[N];
};

}  // namespace

// ---------------------------------------------------------------------------------
// Rotary positions and append.  For pair j of a rotated head, (a, c) -> (a cos t - c sin t,
// a sin t + c cos t) * mscale with t = position * inv_freq[j]; the pair is elements (j, j + rot/2)
// or, interleaved, (2j, 2j + 1); elements rot .. hd - 1 pass.  One rounding, at the store.
//
// The angle is reduced in double, in turns: u = position * inv_freq / 2 pi is off by 2^-52 of at
// most ~2^17 turns for positions below 2^20, so a far position keeps its angle; the remainder to
// the nearest quarter turn (|r| <= 1/8) goes to sincospif in fp32, which is then off by a few
// 2^-25.  A product in fp32 would be wrong in the second digit at position 10^5.
//
// Bound: HBM (every element is read once and written once).  A block takes TOK tokens; their
// sequence, place and sines are worked out once per token for all heads, then each thread moves
// the two 16-byte chunks of a pair group per step.
// ---------------------------------------------------------------------------------
namespace {
constexpr int kRopeThreads = 256;

struct TokInfo {
  long long dst;   // element offset of kv head 0's row in the pages, -1: not appended
  int live;
};
}  // namespace

template <typename QT, typename KT, int TOK, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads) rope_append_paged_kernel(RopeArgs a) {
  __shared__ float2 cs[TOK][64];
  __shared__ TokInfo info[TOK];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, t0 = blockIdx.x * TOK;
  const int nt = min(TOK, a.rows - t0);
  const int half = a.rot >> 1, hd = a.c.hd, Hk = a.c.Hk;
  int seq[TOK];
#pragma unroll
  for (int k = 0; k < TOK; ++k) seq[k] = 0;
  // the sequence of token t: how many row_start[i + 1] are <= t
  for (int i0 = 0; i0 < a.c.batch; i0 += kRopeThreads) {
    const int i = i0 + tid;
    const int end = i < a.c.batch ? a.row_start[i + 1] : 0x7fffffff;
#pragma unroll
    for (int k = 0; k < TOK; ++k) seq[k] += __syncthreads_count(end <= t0 + k);
  }
  for (int k = 0; k < nt; ++k) {
    const int t = t0 + k, b = seq[k];
    const bool live = b < a.c.batch;   // rows behind the last sequence are left as they were
    int place = 0, pos = 0;
    if (live) {
      const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
      place = a.c.lens[b] - (r1 - r0) + (t - r0);
      pos = a.positions ? a.positions[t] : place;
      if (tid == 0) {
        long long dst = -1;
        if (t >= r0 && t < r1 && place >= 0 && place < a.c.capacity()) {
          const int page = a.c.table[(size_t)b * a.c.max_pages + (place >> a.c.page_shift)];
          if (page >= 0 && page < a.c.n_pages)
            dst = page * a.c.page_stride + (long long)(place & (a.c.page() - 1)) * hd;
        }
        if (dst < 0) flag_error(a.c.status, kErrShape);
        info[k].dst = dst;
      }
    }
    if (tid == 0) info[k].live = live;
    for (int j = tid; live && j < half; j += kRopeThreads) {
      const double u = pos * (a.inv_freq[j] * 0.15915494309189533577);   // turns
      const double quarter = rint(4.0 * u);
      float s, c;
      sincospif(2.0f * (float)(u - 0.25 * quarter), &s, &c);
      const int n = (int)((long long)quarter & 3);
      const float cr = n == 0 ? c : n == 1 ? -s : n == 2 ? -c : s;
      const float sr = n == 0 ? s : n == 1 ? c : n == 2 ? -s : -c;
      cs[k][j] = make_float2(cr * a.mscale, sr * a.mscale);
    }
  }
  __syncthreads();

  const int H = a.q ? a.H : 0, heads = H + 2 * Hk;
  KT* const kc = static_cast<KT*>(a.c.k);
  KT* const vc = static_cast<KT*>(a.c.v);
  const long long head_step = (long long)a.c.page() * hd;
  if (VECTOR) {
    constexpr int VEC = 16 / sizeof(QT);
    using In = Pack<QT, VEC>;
    using Out = Pack<KT, VEC>;
    const int per = hd / (2 * VEC);   // pairs of chunks in a head
    const int items = heads * per, turned = a.rot / (2 * VEC);
    for (int it = tid; it < nt * items; it += kRopeThreads) {
      const int k = it / items, rest = it - k * items, h = rest / per, i = rest - h * per;
      if (!info[k].live) continue;
      const int t = t0 + k;
      const bool is_v = h >= H + Hk;
      int e0, e1;
      if (a.interleaved || is_v || i >= turned) {
        e0 = 2 * VEC * i;
        e1 = e0 + VEC;
      } else {
        e0 = VEC * i;
        e1 = e0 + half;
      }
      const QT* src = h < H ? static_cast<const QT*>(a.q) + t * a.ldq + (long long)h * hd
                    : !is_v ? static_cast<const QT*>(a.k) + t * a.ldk + (long long)(h - H) * hd
                            : static_cast<const QT*>(a.v) + t * a.ldv + (long long)(h - H - Hk) * hd;
      const In x0 = *reinterpret_cast<const In*>(src + e0);
      const In x1 = *reinterpret_cast<const In*>(src + e1);
      float y0[VEC], y1[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        y0[e] = to_f<QT>(x0.e[e]);
        y1[e] = to_f<QT>(x1.e[e]);
      }
      if (!is_v) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const int j0 = (e0 + e) >> 1, j1 = (e1 + e) >> 1;
            if (j0 < half) {
              const float2 w = cs[k][j0];
              const float p = y0[e], c = y0[e + 1];
              y0[e] = p * w.x - c * w.y;
              y0[e + 1] = p * w.y + c * w.x;
            }
            if (j1 < half) {
              const float2 w = cs[k][j1];
              const float p = y1[e], c = y1[e + 1];
              y1[e] = p * w.x - c * w.y;
              y1[e + 1] = p * w.y + c * w.x;
            }
          }
        } else if (i < turned) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 w = cs[k][e0 + e];
            const float p = y0[e], c = y1[e];
            y0[e] = p * w.x - c * w.y;
            y1[e] = p * w.y + c * w.x;
          }
        }
      }
      if (h < H) {
        QT* dst = static_cast<QT*>(a.q_out) + t * a.ldo + (long long)h * hd;
        In z0, z1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          z0.e[e] = from_f<QT>(y0[e]);
          z1.e[e] = from_f<QT>(y1[e]);
        }
        *reinterpret_cast<In*>(dst + e0) = z0;
        *reinterpret_cast<In*>(dst + e1) = z1;
      } else if (info[k].dst >= 0) {
        KT* dst = (is_v ? vc + (h - H - Hk) * head_step : kc + (h - H) * head_step) + info[k].dst;
        Out z0, z1;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          z0.e[e] = from_f<KT>(y0[e]);
          z1.e[e] = from_f<KT>(y1[e]);
        }
        *reinterpret_cast<Out*>(dst + e0) = z0;
        *reinterpret_cast<Out*>(dst + e1) = z1;
      }
    }
  } else {
    // odd strides, unaligned rows or half-layout pairs that do not fall on chunks: a thread moves
    // the two elements of a pair (of two passing elements) at a time
    const int per = hd / 2, items = heads * per;
    for (int it = tid; it < nt * items; it += kRopeThreads) {
      const int k = it / items, rest = it - k * items, h = rest / per, i = rest - h * per;
      if (!info[k].live) continue;
      const int t = t0 + k;
      const bool is_v = h >= H + Hk, turn = !is_v && i < half;
      const int e0 = turn && !a.interleaved ? i : 2 * i;
      const int e1 = turn && !a.interleaved ? i + half : 2 * i + 1;
      const QT* src = h < H ? static_cast<const QT*>(a.q) + t * a.ldq + (long long)h * hd
                    : !is_v ? static_cast<const QT*>(a.k) + t * a.ldk + (long long)(h - H) * hd
                            : static_cast<const QT*>(a.v) + t * a.ldv + (long long)(h - H - Hk) * hd;
      float y0 = to_f<QT>(src[e0]), y1 = to_f<QT>(src[e1]);
      if (turn) {
        const float2 w = cs[k][i];
        const float p = y0, c = y1;
        y0 = p * w.x - c * w.y;
        y1 = p * w.y + c * w.x;
      }
      if (h < H) {
        QT* dst = static_cast<QT*>(a.q_out) + t * a.ldo + (long long)h * hd;
        dst[e0] = from_f<QT>(y0);
        dst[e1] = from_f<QT>(y1);
      } else if (info[k].dst >= 0) {
        KT* dst = (is_v ? vc + (h - H - Hk) * head_step : kc + (h - H) * head_step) + info[k].dst;
        dst[e0] = from_f<KT>(y0);
        dst[e1] = from_f<KT>(y1);
      }
    }
  }
}

template <typename QT, typename KT>
static cudaError_t rope_go(const Launch& L, const RopeArgs& a) {
  constexpr int VEC = 16 / sizeof(QT);
  auto off = [&](const void* p, long long ld) { return p && ((reinterpret_cast<uintptr_t>(p) & 15) || ld % VEC != 0); };
  // 16-byte accesses need aligned rows, and half-layout pairs that fall on whole chunks
  const bool vector = !off(a.q, a.ldq) && !off(a.k, a.ldk) && !off(a.v, a.ldv) && !off(a.q ? a.q_out : nullptr, a.ldo) &&
                      (a.interleaved || a.rot % (2 * VEC) == 0);
  constexpr int kMany = 4;
  const bool many = a.rows >= 148 * 8 * kMany;
  const dim3 block(kRopeThreads);
  if (vector) {
    if (many) return launch_k(L, rope_append_paged_kernel<QT, KT, kMany, true>, dim3((a.rows + kMany - 1) / kMany), block, 0, a);
    return launch_k(L, rope_append_paged_kernel<QT, KT, 1, true>, dim3(a.rows), block, 0, a);
  }
  if (many) return launch_k(L, rope_append_paged_kernel<QT, KT, kMany, false>, dim3((a.rows + kMany - 1) / kMany), block, 0, a);
  return launch_k(L, rope_append_paged_kernel<QT, KT, 1, false>, dim3(a.rows), block, 0, a);
}

cudaError_t launch_rope_append_paged(const Launch& L, const RopeArgs& a, int q_elem) {
  if (a.rows <= 0) return cudaSuccess;
  if (q_elem == kF32 && a.c.elem == kF32) return rope_go<float, float>(L, a);
  if (q_elem == kF32 && a.c.elem == kElemF16) return rope_go<float, __half>(L, a);
  if (q_elem == kElemF16 && a.c.elem == kElemF16) return rope_go<__half, __half>(L, a);
  if (q_elem == kBf16 && a.c.elem == kBf16) return rope_go<__nv_bfloat16, __nv_bfloat16>(L, a);
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------------
// Eviction.  Per (sequence, kv head) of length T > keep: the first `first` and last `recent`
// positions stay, and of those between the keep - first - recent of largest weight (ties: the
// lowest index; a NaN counts as largest).
//
// A cluster of CTAs shares a (sequence, kv head).  Each warp takes a contiguous run of the weights and
// holds them in shared memory (up to 20 a lane; what is longer is read again from L2 in each pass).  A radix select over
// the weights' ordered 32-bit keys (four 8-bit digits, the histograms added over distributed shared
// memory; equal digits of a warp are counted together, so that the few distinct leading digits of
// like-sized weights do not serialise on one counter) gives the key of the last one kept and how many of
// its equals stay.  Then the kept positions get their ranks, in order, from the warps' counts, and the
// cluster moves the kept weights and the rows of K and V, 16 bytes a thread, by rank: equal shares
// for the CTAs wherever the kept ones lie.
//
// In place, weights are moved in blocks of ranks that the whole cluster reads before it writes any: a rank
// never exceeds its position, so that a block's writes fall on positions that no later block reads.
//
// Bound: HBM, 2 x kept rows read and written (10.7 and 20.8 us at 64 x 4 x 512 rows of 128 bytes and
// 4 x 8 x 4099 of 256); the select is latency, ~1 us a digit.  One CTA per (sequence, kv head) with a second
// kernel for the rows took 26.9 and 78.4 us, of that the select 14 and 56; this takes 20.2 and 42.0 us (rows
// 9 and 20, a digit 0.6 and, with the cluster's barrier and the sum of its histograms, 2).
// ---------------------------------------------------------------------------------
namespace {
constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32, kEvMaxCluster = 8;
constexpr int kEvHeld = 20;   // weights a thread holds in shared memory
constexpr int kEvRuns = kEvWarps * kEvMaxCluster;

// Keys in the weights' order, all of them between those of a place without a position and of one that stays
// in any case.  -0 counts as 0, a NaN as more than +inf.
constexpr unsigned kKeyNone = 0, kKeyStays = 0xffffffffu;
__device__ __forceinline__ unsigned weight_key(float w) {
  const unsigned u = w != w ? 0x7f800001u : __float_as_uint(w + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
}  // namespace

__global__ void __launch_bounds__(kEvThreads, 2) evict_paged_kernel(EvictArgs a, int row_shift) {
  namespace cg = cooperative_groups;
  __shared__ __align__(16) unsigned hist[4][256];
  __shared__ __align__(16) unsigned total[256];
  __shared__ int picked[4][2];        // of each pass: the digit, how many of its keys are still wanted
  __shared__ unsigned held[kEvHeld][kEvThreads];
  __shared__ int count[2][kEvRuns];   // of every warp of the cluster: kept for sure, equal to the last key
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int unit = blockIdx.x / C, b = unit / a.c.Hk, g = unit - b * a.c.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster.barrier_arrive();   // all CTAs have begun before one writes into another
  for (int i = tid; i < 4 * 256; i += kEvThreads) (&hist[0][0])[i] = 0;
  pdl_wait();
  pdl_trigger();
  const float* w = a.weights + (long long)unit * a.ldw;
  float* wo = a.weights_out + (long long)unit * a.ldwo;
  int* kept = a.kept + (long long)unit * a.keep;
  int T = a.c.lens[b];
  if (T < 0 || T > a.c.capacity()) {
    if (tid == 0) flag_error(a.c.status, kErrShape);
    T = 0;
  }
  const bool cut = T > a.keep;
  const int n = min(T, a.keep);
  const int lo = a.first, hi = T - a.recent;   // where cut: candidates [lo, hi)
  auto weight = [&](int i) { return i < T ? w[i] : 0.f; };
  auto key_of = [&](int i, float x) { return i >= T ? kKeyNone : !cut || i < lo || i >= hi ? kKeyStays : weight_key(x); };

  // this warp's run: kn rows of 32 positions, lane by lane
  const int runs = C * kEvWarps, run = rank * kEvWarps + warp;
  const int kn = (T + 32 * runs - 1) / (32 * runs);
  const int i0 = run * kn * 32 + lane;   // below 2 (T + 32 runs) < 2^31
  for (int k0 = 0; k0 < min(kn, kEvHeld); k0 += 4) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = weight(i0 + 32 * (k0 + k));
#pragma unroll
    for (int k = 0; k < 4; ++k) held[k0 + k][tid] = key_of(i0 + 32 * (k0 + k), x[k]);   // read by this thread alone
  }
  auto each = [&](auto&& f) {
#pragma unroll 4
    for (int k = 0; k < min(kn, kEvHeld); ++k) f(i0 + 32 * k, held[k][tid]);
#pragma unroll 1
    for (int k = kEvHeld; k < kn; ++k) f(i0 + 32 * k, key_of(i0 + 32 * k, weight(i0 + 32 * k)));
  };
  auto sync_all = [&] {   // the cluster's threads; what they wrote is seen
    if (C > 1) cluster.sync();
    else __syncthreads();
  };
  __syncthreads();   // the histograms are zero
  cluster.barrier_wait();

  unsigned key = kKeyStays;
  int equal = n;   // keys above `key` stay, and the first `equal` of its equals
  if (cut) {       // the keep largest; those that stay in any case are among them
    unsigned prefix = 0;
    int left = n;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      if (pass == 0) {
        each([&](int, unsigned u) {
          const unsigned same = __match_any_sync(0xffffffffu, u >> 24);
          if (lane == __ffs(same) - 1) atomicAdd(&hist[0][u >> 24], __popc(same));
        });
      } else {
        each([&](int, unsigned u) {
          if ((u >> (shift + 8)) == prefix) atomicAdd(&hist[pass][(u >> shift) & 255], 1u);
        });
      }
      const unsigned* bins = hist[pass];
      if (C > 1) {
        cluster.sync();
        if (tid < 256) {
          unsigned sum = 0;
#pragma unroll
          for (int r = 0; r < kEvMaxCluster; ++r)
            if (r < C) sum += *cluster.map_shared_rank(&hist[pass][tid], r);
          total[tid] = sum;
        }
        bins = total;
      }
      __syncthreads();
      if (warp == 0) {
        // lane l holds bins 8l .. 8l + 7; from the largest digit down
        const uint4 y = reinterpret_cast<const uint4*>(bins)[2 * lane], z = reinterpret_cast<const uint4*>(bins)[2 * lane + 1];
        const int c[8] = {(int)z.w, (int)z.z, (int)z.y, (int)z.x, (int)y.w, (int)y.z, (int)y.y, (int)y.x};
        int sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += c[k];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_down_sync(0xffffffffu, before, o);
          if (lane + o < 32) before += v;
        }
        before -= sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (before < left && left <= before + c[k]) {   // T > keep: one bin has it
            picked[pass][0] = 8 * lane + 7 - k;
            picked[pass][1] = left - before;
          }
          before += c[k];
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | (unsigned)picked[pass][0];
      left = picked[pass][1];
    }
    key = prefix;
    equal = left;
  }

  // ranks in the order of the positions
  int ns = 0, ne = 0;
  each([&](int, unsigned u) {
    ns += __popc(__ballot_sync(0xffffffffu, u > key));
    ne += __popc(__ballot_sync(0xffffffffu, u == key));
  });
  if (lane < C) {
    int* to = cluster.map_shared_rank(&count[0][0], lane);
    to[run] = ns;
    to[kEvRuns + run] = ne;
  }
  sync_all();
  int rs = 0, re = 0;
#pragma unroll
  for (int k = 0; k < kEvRuns / 32; ++k) {
    const int r = 32 * k + lane;
    if (r < run) {
      rs += count[0][r];
      re += count[1][r];
    }
  }
  rs = __reduce_add_sync(0xffffffffu, rs);
  re = __reduce_add_sync(0xffffffffu, re);
  const unsigned below = (1u << lane) - 1;
  each([&](int i, unsigned u) {
    const bool s = u > key, e = u == key;
    const unsigned bs = __ballot_sync(0xffffffffu, s), be = __ballot_sync(0xffffffffu, e);
    const int nth = re + __popc(be & below);
    if (s || (e && nth < equal)) kept[rs + __popc(bs & below) + min(nth, equal)] = i;
    rs += __popc(bs);
    re += __popc(be);
  });
  sync_all();   // kept is whole (and read past L1: other SMs wrote it)

  // weights
  const bool in_place = wo == w;
  for (int j0 = 0; j0 < n; j0 += C * kEvThreads) {
    const int j = j0 + rank * kEvThreads + tid;
    const float x = j < n ? w[__ldcg(kept + j)] : 0.f;
    if (in_place) sync_all();
    if (j < n) wo[j] = x;
  }
  for (int j = n + rank * kEvThreads + tid; j < a.keep; j += C * kEvThreads) kept[j] = -1;
  for (long long j = n + rank * kEvThreads + tid; j < a.ldwo; j += C * kEvThreads) wo[j] = 0.f;
  if (g == 0 && rank == 0 && tid == 0) a.lens_out[b] = n;

  // rows
  const int per = kEvThreads >> row_shift;            // rows a pass (1 << row_shift chunks of 16 bytes each)
  const int c = tid & ((1 << row_shift) - 1);
  const int mask = a.c.page() - 1;
  const uint4* ks = static_cast<const uint4*>(a.c.k);
  const uint4* vs = static_cast<const uint4*>(a.c.v);
  uint4* kd = static_cast<uint4*>(a.c.k);
  uint4* vd = static_cast<uint4*>(a.c.v);
  const long long page16 = a.c.page_stride * (a.c.elem == kF32 ? 4 : 2) / 16;
  const int* from_table = a.c.table + (long long)b * a.c.max_pages;
  const int* to_table = a.dst_table + (long long)b * a.dst_pages;
  constexpr int U = 4;
  for (int j0 = rank * per * U + (tid >> row_shift); j0 < n; j0 += C * per * U) {
    long long src[U], dst[U];
    uint4 xk[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * per;
      src[u] = -1;
      if (j < n) {
        const int i = __ldcg(kept + j);
        const int sp = from_table[i >> a.c.page_shift], dp = to_table[j >> a.c.page_shift];
        if (sp < 0 || sp >= a.c.n_pages || dp < 0 || dp >= a.c.n_pages) {
          flag_error(a.c.status, kErrShape);
        } else {
          src[u] = sp * page16 + (((long long)g << a.c.page_shift) + (i & mask) << row_shift) + c;
          dst[u] = dp * page16 + (((long long)g << a.c.page_shift) + (j & mask) << row_shift) + c;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0) {
        xk[u] = ks[src[u]];
        xv[u] = vs[src[u]];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0) {
        kd[dst[u]] = xk[u];
        vd[dst[u]] = xv[u];
      }
  }
}

cudaError_t launch_evict_paged(const Launch& L, const EvictArgs& a) {
  const int chunks = a.c.hd * (a.c.elem == kF32 ? 4 : 2) / 16;   // 8, 16 or 32
  const int shift = chunks == 8 ? 3 : chunks == 16 ? 4 : 5;
  const long long units = (long long)a.c.Hk * a.c.batch;
  // more CTAs a unit while two a SM are not reached and each warp has 64 positions
  int C = 1;
  while (C < kEvMaxCluster && units * C < 2 * 148 && a.c.capacity() > C * 2 * kEvThreads) C *= 2;
  return launch_cluster(L, evict_paged_kernel, C, dim3((unsigned)(units * C)), dim3(kEvThreads), 0, a, shift);
}

}  // namespace ms
