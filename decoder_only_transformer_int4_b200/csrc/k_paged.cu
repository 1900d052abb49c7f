// Rotary positions with the append into a paged cache, and eviction from it by accumulated
// attention weight.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <algorithm>
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

// 16 bytes (8 of 16-bit elements made from 4-byte ones) and the values in them, two at a time: one bf16 by the
// conversion instruction runs at a fraction of the rate of a shift or of the conversion of two (measured on
// 4132 rows of 48 heads of 128: 32.7 us against fp16's 22.0).
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T e[N];
};
template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N>& p, float (&y)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = to_f<T>(p.e[e]);
}
template <int N>
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, N>& p, float (&y)[N]) {
  const unsigned* w = reinterpret_cast<const unsigned*>(&p);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    y[e] = __uint_as_float(w[e / 2] << 16);
    y[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
  }
}
template <int N>
__device__ __forceinline__ void pack(Pack<float, N>& p, const float (&y)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) p.e[e] = y[e];
}
template <int N>
__device__ __forceinline__ void pack(Pack<__half, N>& p, const float (&y)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 2) *reinterpret_cast<__half2*>(&p.e[e]) = __floats2half2_rn(y[e], y[e + 1]);
}
template <int N>
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, N>& p, const float (&y)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 2) *reinterpret_cast<__nv_bfloat162*>(&p.e[e]) = __floats2bfloat162_rn(y[e], y[e + 1]);
}

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
// Bound: HBM (every element is read once and written once).  A block takes a few tokens; their
// sequences, places and sines, a chain of three dependent loads and a double-precision reduction, are worked
// out once for all heads.  A thread then has the same two chunks of 16 bytes in every so-manyth head of its
// token, so that its sines stay in registers (read from shared memory for each head, their bank conflicts and
// loads held bf16 rows to half the bandwidth).  32767 rows of 40 heads of 64, fp32 to fp16: 98 us, 6.2 TB/s;
// 4132 rows of 48 bf16 heads of 128: 20.2 us, 5.0 TB/s (the chain at the start shows); 64 rows: 3.1 us.
// ---------------------------------------------------------------------------------
namespace {
constexpr int kRopeThreads = 256, kRopeTokens = 32;

struct TokInfo {
  long long dst;   // element offset of kv head 0's row in the pages, -1: not appended
  int live;
};

// Apart, so that neighbouring threads' 16-byte reads of four fall on all banks (as pairs, 4-way conflicts
// held bf16 rows to half the bandwidth).
struct alignas(16) Sines {
  float c[64], s[64];
};

// A sequence whose rows can be appended: its range lies in the call's rows, its length in the table, and it holds its rows.
// Only such a one is touched at all, as in the attention; a range that is cut off would put rows in places of older ones.
__device__ __forceinline__ bool rope_sequence_ok(const RopeArgs& a, int r0, int r1, int T) {
  return r0 >= 0 && r0 <= r1 && r1 <= a.rows && T <= a.c.capacity() && r1 - r0 <= T;
}

// Sequence, place and sines of the block's tokens; for all its threads, a barrier at the end.
__device__ __forceinline__ void rope_tokens(const RopeArgs& a, int t0, int nt, Sines (&cs)[kRopeTokens], TokInfo (&info)[kRopeTokens]) {
  __shared__ int marks[kRopeTokens], place_of[kRopeTokens];   // position to turn by, of live tokens
  __shared__ bool live_at[kRopeTokens];
  const int tid = threadIdx.x, half = a.rot >> 1;
  // this thread's pair j of every kstep-th token: its frequency is on the way while the tokens are placed
  const int wide = half > 1 ? 1 << (32 - __clz(half - 1)) : 1, j = tid & (wide - 1), kstep = kRopeThreads / wide;
  const double turns = j < half ? a.inv_freq[j] * 0.15915494309189533577 : 0.0;   // per position
  // The sequence of token t: how many row_start[i + 1] are <= t.  Those <= t0 are counted, the others among the
  // block's tokens marked where they end.
  if (tid < kRopeTokens) marks[tid] = 0;
  int b = 0;
  for (int i0 = 0; i0 < a.c.batch; i0 += kRopeThreads) {
    const int i = i0 + tid;
    const bool is = i < a.c.batch;
    const int end = is ? a.row_start[i + 1] : 0;
    // the first block flags the sequences that are left out, whether they have rows or not
    if (blockIdx.x == 0 && is && !rope_sequence_ok(a, a.row_start[i], end, a.c.lens[i])) flag_error(a.c.status, kErrShape);
    b += __syncthreads_count(is && end <= t0);
  }
  if (nt > 1) {
    for (int i = tid; i < a.c.batch; i += kRopeThreads) {
      const int end = a.row_start[i + 1];
      if (end > t0 && end < t0 + nt) atomicAdd(&marks[end - t0], 1);
    }
    __syncthreads();
  }
  int page = -1, place = 0;
  bool live = false;
  if (tid < nt) {
    for (int i = 1; i <= tid; ++i) b += marks[i];
    if (b < a.c.batch) {
      const int t = t0 + tid, r0 = a.row_start[b], r1 = a.row_start[b + 1], T = a.c.lens[b];
      place = T - (r1 - r0) + (t - r0);
      place_of[tid] = a.positions ? a.positions[t] : place;
      // rows before the first sequence and behind the last, and those of a sequence that is left out, stay as they were
      live = rope_sequence_ok(a, r0, r1, T) && t >= r0 && t < r1;
      if (live) page = a.c.table[(size_t)b * a.c.max_pages + (place >> a.c.page_shift)];   // needed at the end
    }
    live_at[tid] = live;
  }
  __syncthreads();
#pragma unroll 2
  for (int k = tid / wide; k < nt; k += kstep) {
    if (j < half && live_at[k]) {
      const double u = place_of[k] * turns;
      const double quarter = rint(4.0 * u);
      float s, c;
      sincospif(2.0f * (float)(u - 0.25 * quarter), &s, &c);
      const int n = (int)((long long)quarter & 3);
      const float cr = n == 0 ? c : n == 1 ? -s : n == 2 ? -c : s;
      const float sr = n == 0 ? s : n == 1 ? c : n == 2 ? -s : -c;
      cs[k].c[j] = cr * a.mscale;
      cs[k].s[j] = sr * a.mscale;
    }
  }
  if (tid < nt) {
    long long dst = -1;
    if (page >= 0 && page < a.c.n_pages) dst = page * a.c.page_stride + (long long)(place & (a.c.page() - 1)) * a.c.hd;
    if (live && dst < 0) flag_error(a.c.status, kErrShape);
    info[tid].dst = dst;
    info[tid].live = live;
  }
  __syncthreads();
}
}  // namespace

namespace {
// N floats of shared memory, aligned to as many
template <int N>
__device__ __forceinline__ void copy_floats(float* to, const float* from) {
  if constexpr (N == 2) {
    const float2 x = *reinterpret_cast<const float2*>(from);
    to[0] = x.x, to[1] = x.y;
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 x = *reinterpret_cast<const float4*>(from + e);
      to[e] = x.x, to[e + 1] = x.y, to[e + 2] = x.z, to[e + 3] = x.w;
    }
  }
}
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a;
  a = x * c - b * s;
  b = x * s + b * c;
}
}  // namespace

template <typename QT, typename KT, bool VECTOR>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_append_paged_kernel(RopeArgs a, int tokens) {
  __shared__ Sines cs[kRopeTokens];
  __shared__ TokInfo info[kRopeTokens];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, t0 = blockIdx.x * tokens;
  const int nt = min(tokens, a.rows - t0);
  const int half = a.rot >> 1, hd = a.c.hd, Hk = a.c.Hk;
  const int H = a.q ? a.H : 0, heads = H + 2 * Hk;
  KT* const kc = static_cast<KT*>(a.c.k);
  KT* const vc = static_cast<KT*>(a.c.v);
  const long long head_step = (long long)a.c.page() * hd;
  auto source = [&](int t, int h) {
    return h < H ? static_cast<const QT*>(a.q) + t * a.ldq + (long long)h * hd
           : h < H + Hk ? static_cast<const QT*>(a.k) + t * a.ldk + (long long)(h - H) * hd
                        : static_cast<const QT*>(a.v) + t * a.ldv + (long long)(h - H - Hk) * hd;
  };
  auto page_row = [&](int k, int h) {
    return (h >= H + Hk ? vc + (h - H - Hk) * head_step : kc + (h - H) * head_step) + info[k].dst;
  };
  if (VECTOR) {
    constexpr int VEC = 16 / sizeof(QT);
    using In = Pack<QT, VEC>;
    using Out = Pack<KT, VEC>;
    // 16-bit chunks hold twice the elements: a second one at once would not fit 64 registers beside the sines (four blocks
    // an SM; 4132 bf16 rows of 48 heads: 26.1 us, 21.8 with one)
    constexpr int U = sizeof(QT) == 2 ? 1 : 2;
    // a thread has the same two chunks of every head_groups-th head of one token, and their sines in registers
    const int shift = hd == 64 ? (VEC == 4 ? 3 : 2) : (VEC == 4 ? 4 : 3);   // 2^shift pairs of chunks in a head
    const int i = tid & ((1 << shift) - 1), head_groups = (kRopeThreads >> shift) / tokens;   // tokens: a power of two
    const int slot = tid >> shift, k = slot / head_groups, h0 = slot - k * head_groups;
    const int turned = a.rot / (2 * VEC);
    const bool mine = k < nt;
    // q and k heads: chunks e0, e1; v heads, which pass: f0, f1
    const int f0 = VEC * i, f1 = f0 + hd / 2;
    const int e0 = a.interleaved || i < turned ? f0 : a.rot + VEC * (i - turned);
    const int e1 = a.interleaved ? f1 : e0 + (i < turned ? half : (hd - a.rot) / 2);
    float c[VEC], s[VEC];
    int n0 = 0, n1 = 0;   // interleaved: pairs of the two chunks that turn; else of both together
    rope_tokens(a, t0, nt, cs, info);
    if (a.interleaved) {
      n0 = min(max(half - e0 / 2, 0), VEC / 2);
      n1 = min(max(half - e1 / 2, 0), VEC / 2);
      copy_floats<VEC / 2>(c, cs[k].c + e0 / 2);
      copy_floats<VEC / 2>(s, cs[k].s + e0 / 2);
      copy_floats<VEC / 2>(c + VEC / 2, cs[k].c + e1 / 2);
      copy_floats<VEC / 2>(s + VEC / 2, cs[k].s + e1 / 2);
    } else if (i < turned) {
      n0 = VEC;
      copy_floats<VEC>(c, cs[k].c + e0);
      copy_floats<VEC>(s, cs[k].s + e0);
    }
    if (!mine || !info[k].live) return;
    for (int h1 = h0; h1 < heads; h1 += U * head_groups) {
      In x0[U], x1[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h1 + u * head_groups;
        if (h < heads) {
          const QT* src = source(t0 + k, h);
          x0[u] = *reinterpret_cast<const In*>(src + (h < H + Hk ? e0 : f0));
          x1[u] = *reinterpret_cast<const In*>(src + (h < H + Hk ? e1 : f1));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h1 + u * head_groups;
        if (h < heads) {
          const bool is_v = h >= H + Hk;
          float y0[VEC], y1[VEC];
          unpack(x0[u], y0);
          unpack(x1[u], y1);
          if (!is_v) {
            if (a.interleaved) {
#pragma unroll
              for (int e = 0; e < VEC / 2; ++e) {
                if (e < n0) turn(y0[2 * e], y0[2 * e + 1], c[e], s[e]);
                if (e < n1) turn(y1[2 * e], y1[2 * e + 1], c[VEC / 2 + e], s[VEC / 2 + e]);
              }
            } else if (n0) {
#pragma unroll
              for (int e = 0; e < VEC; ++e) turn(y0[e], y1[e], c[e], s[e]);
            }
          }
          if (h < H) {
            QT* dst = static_cast<QT*>(a.q_out) + (t0 + k) * a.ldo + (long long)h * hd;
            In z0, z1;
            pack(z0, y0);
            pack(z1, y1);
            *reinterpret_cast<In*>(dst + e0) = z0;
            *reinterpret_cast<In*>(dst + e1) = z1;
          } else if (info[k].dst >= 0) {
            KT* dst = page_row(k, h);
            Out z0, z1;
            pack(z0, y0);
            pack(z1, y1);
            *reinterpret_cast<Out*>(dst + (is_v ? f0 : e0)) = z0;
            *reinterpret_cast<Out*>(dst + (is_v ? f1 : e1)) = z1;
          }
        }
      }
    }
  } else {
    // odd strides, unaligned rows or half-layout pairs that do not fall on chunks: a thread moves
    // the two elements of a pair (of two passing elements) at a time (the sizes above with pairs of 30 elements: 205 and 82 us,
    // floors 93 and 17)
    rope_tokens(a, t0, nt, cs, info);
    const int per = hd / 2, items = heads * per;
    for (int it = tid; it < nt * items; it += kRopeThreads) {
      const int k = it / items, rest = it - k * items, h = rest / per, i = rest - h * per;
      if (!info[k].live) continue;
      const bool turned = h < H + Hk && i < half;
      const int e0 = turned && !a.interleaved ? i : 2 * i;
      const int e1 = turned && !a.interleaved ? i + half : 2 * i + 1;
      const QT* src = source(t0 + k, h);
      float y0 = to_f<QT>(src[e0]), y1 = to_f<QT>(src[e1]);
      if (turned) turn(y0, y1, cs[k].c[i], cs[k].s[i]);
      if (h < H) {
        QT* dst = static_cast<QT*>(a.q_out) + (t0 + k) * a.ldo + (long long)h * hd;
        dst[e0] = from_f<QT>(y0);
        dst[e1] = from_f<QT>(y1);
      } else if (info[k].dst >= 0) {
        KT* dst = page_row(k, h);
        dst[e0] = from_f<KT>(y0);
        dst[e1] = from_f<KT>(y1);
      }
    }
  }
}

template <typename QT, typename KT>
static cudaError_t rope_go(const Launch& L, const RopeArgs& a, int n_sm) {
  constexpr int VEC = 16 / sizeof(QT);
  auto off = [&](const void* p, long long ld) { return p && ((reinterpret_cast<uintptr_t>(p) & 15) || ld % VEC != 0); };
  // 16-byte accesses need aligned rows, and half-layout pairs that fall on whole chunks
  const bool vector = !off(a.q, a.ldq) && !off(a.k, a.ldk) && !off(a.v, a.ldv) && !off(a.q ? a.q_out : nullptr, a.ldo) &&
                      (a.interleaved || a.rot % (2 * VEC) == 0);
  // Tokens a block, a power of two: more of them share the chain.  Two for each thread to move at least, where that leaves
  // two blocks an SM (27600 rows of 3 heads: 13.7 us at 32 tokens, 26.3 at 8); up to 8 while 1.5 waves of blocks are
  // left to overlap one block's chain with another's copies (4132 rows of 48 heads: 26.7 us at 8, 25.2 at 4; 32767 of 40: 98 at
  // 8, 103 at 4, 105 at 16).
  int tokens = 1;
  const int items = ((a.q ? a.H : 0) + 2 * a.c.Hk) * a.c.hd / (vector ? 2 * VEC : 2), most = std::min(kRopeTokens, kRopeThreads * 2 * VEC / a.c.hd);
  while (tokens < most && a.rows >= (long long)n_sm * 2 * 2 * tokens && (tokens * items < 2 * kRopeThreads || (tokens < 8 && a.rows >= (long long)n_sm * 6 * 2 * tokens))) tokens *= 2;
  // or as many as make one wave of all blocks, each with 24 items a thread at most (3000 rows of 72 heads: 10% faster at 8
  // than at 2)
  int wave = 1;
  while (wave < most && a.rows > (long long)n_sm * 4 * wave) wave *= 2;
  if (a.rows <= (long long)n_sm * 4 * wave && wave * items <= 24 * kRopeThreads) tokens = std::max(tokens, wave);
  const dim3 grid((a.rows + tokens - 1) / tokens), block(kRopeThreads);
  if (vector) return launch_k(L, rope_append_paged_kernel<QT, KT, true>, grid, block, 0, a, tokens);
  return launch_k(L, rope_append_paged_kernel<QT, KT, false>, grid, block, 0, a, tokens);
}

cudaError_t launch_rope_append_paged(const Launch& L, const RopeArgs& a, int q_elem, int n_sm) {
  if (a.rows <= 0) return cudaSuccess;
  if (q_elem == kF32 && a.c.elem == kF32) return rope_go<float, float>(L, a, n_sm);
  if (q_elem == kF32 && a.c.elem == kElemF16) return rope_go<float, __half>(L, a, n_sm);
  if (q_elem == kElemF16 && a.c.elem == kElemF16) return rope_go<__half, __half>(L, a, n_sm);
  if (q_elem == kBf16 && a.c.elem == kBf16) return rope_go<__nv_bfloat16, __nv_bfloat16>(L, a, n_sm);
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------------
// Eviction.  Per (sequence, kv head) of length T > keep: the first `first` and last `recent`
// positions stay, and of those between the keep - first - recent of largest weight (ties: the
// lowest index; a NaN counts as largest).
//
// A cluster of CTAs shares a (sequence, kv head).  Each warp takes a contiguous run of the weights and
// holds their keys in shared memory (up to 16 a lane; what is longer is read again from L2 in each pass).  A radix select over
// the weights' ordered 32-bit keys (8-bit digits, the histograms added over distributed shared
// memory; equal leading digits of a warp are counted together, so that the few distinct ones of
// like-sized weights do not serialise on one counter) narrows down the key of the last one kept; as soon as at most
// 128 keys are left for it, every CTA gets them all and ranks them by comparing each with each.  That gives the key and how
// many of its equals stay.  Then the kept positions get their ranks, in order, from the warps' counts, and the
// cluster moves the kept weights and the rows of K and V, 16 bytes a thread, by rank: equal shares
// for the CTAs wherever the kept ones lie.
//
// In place, weights are moved in blocks of ranks that the whole cluster reads before it writes any: a rank
// never exceeds its position, so that a block's writes fall on positions that no later block reads.
//
// Bound: HBM, 2 x kept rows read and written (10.7 and 20.8 us at 64 x 4 x 512 rows of 128 bytes and
// 4 x 8 x 4099 of 256); the select is latency: a digit takes 0.6 us in one CTA, 2 to 2.4 in a cluster (its barrier 0.9, the sum of
// its histograms 0.5).  20.9 and 39 us; all four digits 20.5 and 41.2; one CTA per (sequence, kv head) with a second
// kernel for the rows 26.9 and 78.4, of that the select 14 and 56.  Moving the rows that stay in any case while the barriers are
// waited for did not pay (21.8 and 44.5): their loads delay the select's.
// ---------------------------------------------------------------------------------
namespace {
constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32, kEvMaxCluster = 8;
constexpr int kEvHeld = 16;   // weights a thread holds in shared memory
constexpr int kEvFew = 128;   // so few candidates for the last place are ranked by comparing all with all
constexpr int kEvRuns = kEvWarps * kEvMaxCluster;

// Keys in the weights' order, all of them between those of a place without a position and of one that stays
// in any case.  -0 counts as 0, a NaN as more than +inf.
constexpr unsigned kKeyNone = 0, kKeyStays = 0xffffffffu;
__device__ __forceinline__ unsigned weight_key(float w) {
  const unsigned u = w != w ? 0x7f800001u : __float_as_uint(w + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Rows of K and V of one (sequence, kv head) by rank: this block's share of the n of them, `blocks` blocks of kEvThreads in all.
__device__ __forceinline__ void move_rows(const EvictArgs& a, int row_shift, int b, int g, int n, int block, int blocks) {
  const int tid = threadIdx.x;
  const int* kept = a.kept + ((long long)b * a.c.Hk + g) * a.keep;
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
  for (int j0 = block * per * U + (tid >> row_shift); j0 < n; j0 += blocks * per * U) {
    long long src[U], dst[U];
    uint4 xk[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * per;
      src[u] = -1;
      if (j < n) {
        const int i = __ldcg(kept + j), to = j >> a.c.page_shift;
        const int sp = from_table[i >> a.c.page_shift], dp = to < a.dst_pages ? to_table[to] : -1;
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

}  // namespace

__global__ void __launch_bounds__(kEvThreads, 2) evict_paged_kernel(EvictArgs a, int row_shift, int rows_here) {
  namespace cg = cooperative_groups;
  __shared__ __align__(16) unsigned hist[4][256];
  __shared__ __align__(16) unsigned total[256];
  __shared__ int picked[4][3];        // of each pass: the digit, how many of its keys are still wanted, how many there are
  __shared__ __align__(16) unsigned few[kEvFew];
  __shared__ unsigned last_key;
  __shared__ int last_equal, few_count;   // few_count: the first CTA's counts for all
  __shared__ unsigned held[kEvHeld][kEvThreads];
  __shared__ int count[2][kEvRuns];   // of every warp of the cluster: kept for sure, equal to the last key
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int unit = blockIdx.x / C, b = unit / a.c.Hk, g = unit - b * a.c.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster.barrier_arrive();   // all CTAs have begun before one writes into another
  for (int i = tid; i < 4 * 256; i += kEvThreads) (&hist[0][0])[i] = 0;
  if (tid < kEvFew) few[tid] = kKeyNone;
  if (tid == 0) few_count = 0;
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
  constexpr int kAtOnce = 8;
  static_assert(kEvHeld % kAtOnce == 0, "");
  for (int k0 = 0; k0 < min(kn, kEvHeld); k0 += kAtOnce) {
    float x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) x[k] = weight(i0 + 32 * (k0 + k));
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) held[k0 + k][tid] = key_of(i0 + 32 * (k0 + k), x[k]);   // read by this thread alone
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
            picked[pass][2] = c[k];
          }
          before += c[k];
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | (unsigned)picked[pass][0];
      left = picked[pass][1];
      if (pass == 3) {
        key = prefix;
        equal = left;
      } else if (picked[pass][2] <= kEvFew) {
        // every CTA gets them all, in any order
        each([&](int, unsigned u) {
          if ((u >> shift) == prefix) {
            const int at = atomicAdd(cluster.map_shared_rank(&few_count, 0), 1);
            for (int r = 0; r < C; ++r) cluster.map_shared_rank(few, r)[at] = u;
          }
        });
        sync_all();
        if (tid < picked[pass][2]) {
          const unsigned u = few[tid];
          int above = 0, same = 0;
#pragma unroll 4
          for (int j = 0; j < picked[pass][2]; j += 4) {   // behind the last one: kKeyNone, below all
            const uint4 x = *reinterpret_cast<const uint4*>(few + j);
            above += (x.x > u) + (x.y > u) + (x.z > u) + (x.w > u);
            same += (x.x == u) + (x.y == u) + (x.z == u) + (x.w == u);
          }
          if (above < left && left <= above + same) {   // the same for all equal ones
            last_key = u;
            last_equal = left - above;
          }
        }
        __syncthreads();
        key = last_key;
        equal = last_equal;
        break;
      }
    }
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

  if (rows_here) move_rows(a, row_shift, b, g, n, rank, C);
}

__global__ void __launch_bounds__(kEvThreads, 2) evict_rows_kernel(EvictArgs a, int row_shift) {
  pdl_wait();
  pdl_trigger();
  move_rows(a, row_shift, blockIdx.z, blockIdx.y, a.lens_out[blockIdx.z], blockIdx.x, gridDim.x);
}

cudaError_t launch_evict_paged(const Launch& L, const EvictArgs& a, int n_sm) {
  const int chunks = a.c.hd * (a.c.elem == kF32 ? 4 : 2) / 16;   // 8, 16 or 32
  const int shift = chunks == 8 ? 3 : chunks == 16 ? 4 : 5;
  const long long units = (long long)a.c.Hk * a.c.batch;
  // More CTAs a unit, up to two an SM, while each has 64 positions a warp or 128 KB of rows.  Few units want many CTAs for
  // their rows (12 units of 1310 fp32 rows of 128: 17 us in clusters of 8, 34 in pairs), small ones are faster without the
  // cluster's barriers (52 units of 170 rows of 256 bytes: 9.6 us alone, 13.8 in fours).
  const long long bytes = (long long)std::min(a.keep, a.c.capacity()) * chunks * 16 * 2;
  int C = 1;
  while (C < kEvMaxCluster && units * C * 2 <= 2 * n_sm && (bytes > C * (128ll << 10) || a.c.capacity() > C * 2 * kEvThreads)) C *= 2;
  // Fewer CTAs than SMs with much to move: the rows get a grid of their own (4 units of 14191 fp32 rows of 128: 37 us,
  // 93 where the clusters move them).
  const bool apart = units * C < n_sm && bytes > C * (256ll << 10);
  const cudaError_t e = launch_cluster(L, evict_paged_kernel, C, dim3((unsigned)(units * C)), dim3(kEvThreads), 0, a, shift, apart ? 0 : 1);
  if (e != cudaSuccess || !apart) return e;
  const int at_once = (kEvThreads >> shift) * 4;
  const int blocks = std::min<long long>((std::min(a.keep, a.c.capacity()) + at_once - 1) / at_once, 4 * n_sm / units + 1);
  return launch_k(L, evict_rows_kernel, dim3(blocks, a.c.Hk, a.c.batch), dim3(kEvThreads), 0, a, shift);
}

}  // namespace ms
