// Rotary positions with the append into a paged cache, and eviction from it by accumulated
// attention weight.
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
// lowest index; a NaN counts as largest).  Two kernels:
//
// evict_select_kernel, one CTA per (sequence, kv head): a radix select over the weights' ordered
// 32-bit keys (four 8-bit digits; equal digits of a warp are counted together, so that the few
// distinct leading digits of like-sized weights do not serialise on one counter) gives the key of
// the last one kept and how many of its equals stay; then one ordered pass writes the kept indexes
// and their weights by rank.  The weights may be compacted in place: a rank never exceeds its
// position, and a chunk is read before any of it is written.
//
// evict_move_kernel copies the kept rows of K and V into the sequence's new pages, 16 bytes a
// thread, in the order of their positions.  Bound: HBM, 2 x kept rows read and written.
// ---------------------------------------------------------------------------------
namespace {
constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

__device__ __forceinline__ unsigned weight_key(float w) {
  unsigned u = w != w ? 0x7fffffffu : __float_as_uint(w + 0.0f);   // -0 counts as 0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
}  // namespace

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ unsigned hist[256];
  __shared__ unsigned pick[2];          // digit chosen, how many of its keys are still wanted
  __shared__ unsigned wsum[32];
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = (long long)b * a.c.Hk + g;
  const float* w = a.weights + row * a.ldw;
  float* wo = a.weights_out + row * a.ldwo;
  int* kept = a.kept + row * a.keep;
  int T = a.c.lens[b];
  if (T < 0 || T > a.c.capacity() || T > a.ldw) {
    if (tid == 0) flag_error(a.c.status, kErrShape);
    T = 0;
  }
  const bool cut = T > a.keep;
  const int lo = cut ? a.first : 0, hi = cut ? T - a.recent : 0;   // candidates [lo, hi)
  const unsigned want = cut ? a.keep - a.first - a.recent : 0;
  unsigned key = 0xffffffffu, equal = 0;   // keys above `key` stay, and the first `equal` of its equals
  if (want) {
    unsigned prefix = 0, left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int i0 = lo; i0 < hi; i0 += kSelThreads) {
        const int i = i0 + tid;
        unsigned d = 256;
        if (i < hi) {
          const unsigned u = weight_key(w[i]);
          if (shift == 24 || (u >> (shift + 8)) == prefix) d = (u >> shift) & 255;
        }
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (d < 256 && lane == __ffs(same) - 1) atomicAdd(&hist[d], __popc(same));
      }
      __syncthreads();
      if (warp == 0) {
        // bins from the largest digit down: lane l holds bins 255 - 8l .. 248 - 8l
        unsigned c[8], sum = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += c[k] = hist[255 - 8 * lane - k];
        unsigned before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        before -= sum;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (before < left && left <= before + c[k]) {
            pick[0] = 255 - 8 * lane - k;
            pick[1] = left - before;
          }
          before += c[k];
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | pick[0];
      left = pick[1];
      __syncthreads();
    }
    key = prefix;
    equal = left;
  }
  // ranks in the order of the positions, four consecutive positions a thread; counts of sure ones
  // in the low half of a word, of equals in the high half (a chunk has 4096 positions)
  unsigned sure0 = 0, eq0 = 0;
  for (int i0 = 0; i0 < T; i0 += 4 * kSelThreads) {
    float v[4];
    unsigned mine = 0, flags = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + 4 * tid + k;
      v[k] = i < T ? w[i] : 0.f;
      if (i < T) {
        const unsigned u = weight_key(v[k]);
        const bool inside = cut && i >= lo && i < hi;
        if (!inside || (want && u > key)) {
          mine += 1u;
          flags |= 1u << k;
        } else if (want && u == key) {
          mine += 1u << 16;
          flags |= 16u << k;
        }
      }
    }
    unsigned incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    unsigned base = 0, all = 0;
    {
      const unsigned x = wsum[lane];
      unsigned y = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
      }
      base = __shfl_sync(0xffffffffu, y - x, warp);
      all = __shfl_sync(0xffffffffu, y, 31);
    }
    base += incl - mine;
    unsigned sure = sure0 + (base & 0xffffu), eq = eq0 + (base >> 16);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool s = flags & (1u << k), e = flags & (16u << k);
      if (s || (e && eq < equal)) {
        const unsigned r = sure + min(eq, equal);
        kept[r] = i0 + 4 * tid + k;
        wo[r] = v[k];
      }
      sure += s;
      eq += e;
    }
    sure0 += all & 0xffffu;
    eq0 += all >> 16;
  }
  __syncthreads();
  const int n = min(T, a.keep);
  for (int i = n + tid; i < a.keep; i += kSelThreads) kept[i] = -1;
  for (long long i = n + tid; i < a.ldwo; i += kSelThreads) wo[i] = 0.f;
  if (g == 0 && tid == 0) a.lens_out[b] = n;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, int row_shift) {
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.y, b = blockIdx.z;
  const int per = kMoveThreads >> row_shift;            // rows a pass (1 << row_shift chunks of 16 bytes each)
  const int c = threadIdx.x & ((1 << row_shift) - 1);
  const int* kept = a.kept + ((long long)b * a.c.Hk + g) * a.keep;
  const int mask = a.c.page() - 1;
  const uint4* ks = static_cast<const uint4*>(a.c.k);
  const uint4* vs = static_cast<const uint4*>(a.c.v);
  uint4* kd = static_cast<uint4*>(a.c.k);
  uint4* vd = static_cast<uint4*>(a.c.v);
  const long long page16 = a.c.page_stride * (a.c.elem == kF32 ? 4 : 2) / 16;
  constexpr int U = 4;
  const int j0 = blockIdx.x * per * U + (threadIdx.x >> row_shift);
  long long src[U], dst[U];
  uint4 xk[U], xv[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = j0 + u * per;
    src[u] = -1;
    if (j < a.keep) {
      const int i = kept[j];
      if (i >= 0) {
        const int sp = a.c.table[(long long)b * a.c.max_pages + (i >> a.c.page_shift)];
        const int dp = a.dst_table[(long long)b * a.dst_pages + (j >> a.c.page_shift)];
        if (sp < 0 || sp >= a.c.n_pages || dp < 0 || dp >= a.c.n_pages) {
          flag_error(a.c.status, kErrShape);
        } else {
          src[u] = sp * page16 + (((long long)g << a.c.page_shift) + (i & mask) << row_shift) + c;
          dst[u] = dp * page16 + (((long long)g << a.c.page_shift) + (j & mask) << row_shift) + c;
        }
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

cudaError_t launch_evict_paged(const Launch& L, const EvictArgs& a) {
  cudaError_t e = launch_k(L, evict_select_kernel, dim3(a.c.Hk, a.c.batch), dim3(kSelThreads), 0, a);
  if (e != cudaSuccess) return e;
  const int chunks = a.c.hd * (a.c.elem == kF32 ? 4 : 2) / 16;   // 8, 16 or 32
  const int shift = chunks == 8 ? 3 : chunks == 16 ? 4 : 5;
  const int rows = (kMoveThreads >> shift) * 4;
  return launch_k(L, evict_move_kernel, dim3((a.keep + rows - 1) / rows, a.c.Hk, a.c.batch), dim3(kMoveThreads), 0, a,
                  shift);
}

}  // namespace ms
