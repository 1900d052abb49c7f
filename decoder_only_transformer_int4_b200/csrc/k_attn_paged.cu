// Attention of the newest rows of each sequence over a paged KV cache.
//
// Row i of the n newest of a sequence of length T sees positions t < T - n + 1 + i:
//   o_i = sum_t p_it v_t,  p_it = exp(scale q_i.k_t) / sum_t' exp(scale q_i.k_t'),
// query head h reading kv head h / (H / Hk).  Optionally w[g][t] += sum of p_it over the rows and the
// heads of group g.
//
// Bound: HBM, every K and V row of a sequence is read once for all heads of its group and all newest
// rows, up to 32 at a time, 16 with an fp32 cache (2 T Hk hd elements a pass).  One cache of 131071 positions (8 kv heads of 64, fp16) takes 48 us with
// the join, 5.5 TB/s; 16 ragged sequences of up to 16411 (8 heads of 128, bf16) 98 us at one row each (6.1 TB/s)
// and 115 us at up to six (5.7 TB/s while the first kernel runs), where a tile of 24 rows costs about as many issue slots as the
// memory leaves.  64 sequences of 505 to 1024 take 18.0 us (19.8 with weights) for 52 MB: 4.5 us until the first tile is
// there, then seven tiles a CTA, then the join.
//
// The products stay on warp-level MMAs: S^T = K Q^T and O^T = V^T P^T, sixteen cached positions (or elements
// of a head) on the M side, rows in tiles of 8 on the N side, so that the 3 or 4 rows of a decoding group pad to 8.
// A tcgen05 variant for more than 16 rows (128 positions a tile, one to a TMEM lane, sums in TMEM) was built and left out: 200 us
// against 115 on the case above, 100 against 83 at 56 rows.  It moved its tiles with cp.async through the load-store path, a third
// of its time a tile, and one group of eight softmax warps worked in step; with TMA copies it has not been tried.
//
// Split.  The positions of all (sequence, kv head, row tile) units are cut into tiles of 64 and laid
// end to end; every resident CTA takes an equal run of tiles, whatever the lengths.  A run crosses
// units: a unit that lies in one CTA is finished there, a cut one leaves (m, l, o) partials, one slot
// for the piece that begins a CTA's run and one for the piece that ends it, which attn_finish_kernel adds.
// Nothing waits for another CTA, no counter has to be cleared, and the order of every sum is fixed.
// A call whose units all fit the GPU as clusters with at most two tiles to a CTA (1024 positions) joins over
// distributed shared memory instead, in one launch: one fp32 stream of 577 positions 6.7 us, 9.5 in two kernels; with eight
// tiles to a CTA (4000 positions) the cluster's 14.1 us lose to 8.8.
//
// Inside a CTA each warp takes its own 16 positions of every tile and streams them with cp.async
// through its own ring, so the warps meet only at a unit's end.  16 positions lie within one page (a
// page holds a power of two of at least 16 positions), so a step needs one table entry; the entries of
// the next 16 tiles are looked up at once, one per lane.  Two to three CTAs share an SM: with one, four warps
// cannot hide a step's chain of loads, products and exponentials (drafted rows: 211 us).
//
// Arithmetic.  16-bit caches: products of m16n8k16 with fp32 sums; the probabilities enter P V as a
// 16-bit pair hi + lo (two MMAs), so that they carry 16 (bf16) or up to 22 (fp16) bits and not 8 or 11: the
// error of the result is then the rounding of its store.  fp16 pairs have a range: where the result is fp16, too, what
// is lost of a probability is at most 2^-35 of its row's largest (so one below that counts as 0, which shows where the v of
// all larger ones are next to 0); where it is fp32, small probabilities are brought into the range by powers of two, step by
// step, and keep their 22 bits whatever leads them.  fp32 queries on a half cache enter as a pair
// too, after an exact power-of-two scale of the row.  fp32 caches: m16n8k8 tf32 with every operand as a
// pair of 11-bit halves, three products (hi hi, hi lo, lo hi): ~2^-21 per product.  Running maximum and
// sum in fp32, in the exponent's base 2.  Where the result is stored in fp32, each step's P V is summed
// from zero and added to the running sum by a rounded addition: the tensor cores cut their sums off, which
// over 3000 positions added up to three times the plain fp32 form's error.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <algorithm>
#include <atomic>
#include <type_traits>
#include "ms_device.cuh"
#include "ms_launch.cuh"
#include "ms_paged.h"

namespace ms {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStep = 16;                  // positions a warp takes at a time
constexpr int kTile = kStep * kWarps;      // positions of a tile
constexpr int kMaxCluster = 8;            // CTAs that share a unit
constexpr int kClusterTiles = 2;          // the most tiles each of them takes
constexpr int kRing = 32;                  // tile descriptors a warp holds (two halves of 16)

struct Desc {
  long long off;         // element offset of the 16 positions' first row in the pages, -1: no page there
  int pos0;              // first position
  int row0;              // first row of the row tile
  short b, kvh;          // sequence, kv head
  short nvalid;          // positions of the 16 that exist
  short ends;            // bits 0, 1: this tile begins the CTA's piece, the unit; bits 2, 3: ends the piece, the unit
};

struct Kargs {
  PagedView c;
  const void* q;
  void* out;
  long long ldq, ldo;
  const int* row_start;
  int rows, max_rows, hpg, rb;      // rb: the most row tiles a (sequence, kv head) may have
  float scale2;                     // scale * log2(e)
  float* part;                      // [CTAs][2][R][hd] unscaled sums of cut units
  float2* ml;                       // [CTAs][2][R] their (max, sum)
  float* scores;                    // [batch][Hk][hpg * max_rows][capacity], or null
  float2* stats;                    // [batch][Hk][hpg * max_rows] final (max, sum), with scores
  int grid;                         // CTAs of the main kernel
  int cluster;                      // CTAs that share a unit, 0: runs of tiles
  int slices;                       // CTAs that join a unit's pieces
};

// The exponent of every probability is raised by this where P enters as fp16 pairs, so that fewer of them fall
// among the subnormal halves; it cancels in o / l.
template <typename KT>
constexpr float bias_of() { return std::is_same<KT, __half>::value ? 10.f : 0.f; }
// fp32 results from a half cache: lo enters 2^12 times as large and its sum is scaled back.  The pair of a probability from
// 2^-14 to 2^14 (the normal halves) is then off by 2^-22 of it: lo's step of 2^-24 counts 2^-36.  Smaller ones are brought
// into that range before.  64 streams 19.8 us, 19.2 without; 5% with several rows.
constexpr float kLoUp = 4096.f, kPairFrom = 0x1p-14f;
// How far a score may pass the running reference before sums are scaled anew: probabilities stay below 2^14
constexpr float kSlack = 4.f;

template <typename KT, bool Q32, int HD, int NB>
struct Shape {
  static constexpr bool kF32 = sizeof(KT) == 4;
  static constexpr int R = 8 * NB;
  static constexpr int kRowBytes = HD * sizeof(KT);
  static constexpr int kStageBytes = 2 * kStep * kRowBytes;      // K then V of one warp's step
  // 16 KB (fp32, 128 elements): one stage and two CTAs an SM instead of two stages and one CTA
  // (67 sequences of 20 heads on 5: 37 us, 48 with two stages)
  static constexpr int kStages = kStageBytes <= 4096 ? 3 : kStageBytes <= 8192 ? 2 : 1;
  static constexpr int kQBytes = R * HD * ((kF32 || Q32) ? 4 : 2);   // Q32 on halves: hi and lo planes
  static constexpr bool kQRegs = !kF32 && NB * (HD / 16) * (Q32 ? 2 : 1) <= 16;   // Q's fragments stay in registers
  static constexpr int kObufStride = HD + 4;
  static constexpr int kBufs = HD == 64 && NB <= 2 ? kWarps : 1;   // buffers of the merge: one a warp, or one in turn
  static constexpr int kObufBytes = kBufs * R * kObufStride * 4;
  static constexpr int kDescBytes = kWarps * kRing * (int)sizeof(Desc);
  static constexpr int kSmall = R * 4 * (2 + 2 * kWarps + 2);
  static constexpr int kFixed = kWarps * kStages * kStageBytes + kQBytes + kObufBytes + kDescBytes + kSmall;
  static size_t smem(int batch) { return kFixed + 4 * (size_t)(batch + 1); }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the same, or 16 zero bytes where !take (nothing is read then)
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2^x to 2 ulp; results below the smallest normal number are 0
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two fp32 multiplications, or multiplications and additions, in one instruction: (a, b) *= f, and (a, b) += (x, y) * (f, g)
__device__ __forceinline__ void mul2(float& a, float& b, float f) {
  asm("{.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %2};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;}"
      : "+f"(a), "+f"(b) : "f"(f));
}
__device__ __forceinline__ void fma2(float& a, float& b, float x, float y, float f, float g) {
  asm("{.reg .b64 p, q, r;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\tfma.rn.f32x2 p, q, r, p;\n\tmov.b64 {%0, %1}, p;}"
      : "+f"(a), "+f"(b) : "f"(x), "f"(y), "f"(f), "f"(g));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// the 8 x 8 matrix of 16-bit elements that a warp holds, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename KT>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi is x rounded to 11 significant bits (half away from zero), lo the exact difference, of
// which the product uses 11 bits.  Cut off instead of rounded, hi would leave a lo of up to twice the size
// and always x's sign: the dropped lo lo and the cut of lo would then add up over a row (measured: 2.5 times
// the error of the result).
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

template <typename T> __device__ __forceinline__ float as_float(T x);
template <> __device__ __forceinline__ float as_float<float>(float x) { return x; }
template <> __device__ __forceinline__ float as_float<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T rounded(float x);
template <> __device__ __forceinline__ float rounded<float>(float x) { return x; }
template <> __device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// a, b as a pair of the 16-bit type, and what the rounding left of them
template <typename KT> struct Two;
template <> struct Two<__half> {
  static __device__ __forceinline__ uint32_t pack(float a, float b, float& ra, float& rb) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    ra = a - f.x;
    rb = b - f.y;
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <> struct Two<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float a, float b, float& ra, float& rb) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
    ra = a - __uint_as_float(w << 16);   // (the conversion instruction is slower than a shift)
    rb = b - __uint_as_float(w & 0xffff0000u);
    return w;
  }
};

template <typename KT>
__device__ __forceinline__ float staged(const unsigned char* p) { return as_float<KT>(*reinterpret_cast<const KT*>(p)); }

// Chunk (16 bytes) c of row r of a staged K or V step.  16-bit: the 8 rows of an ldmatrix fall on all
// banks.  fp32 K: lanes read rows 2i, 2i + 1 at four chunks each; fp32 V: rows 2t at two chunks each.
template <bool F32>
__device__ __forceinline__ int swz_k(int c, int r) { return F32 ? c ^ ((r & 1) << 2) : c ^ (r & 7); }
template <bool F32>
__device__ __forceinline__ int swz_v(int c, int r) { return F32 ? c ^ (((r >> 1) & 3) << 1) : c ^ (r & 7); }

// Row range and length of sequence b; rows n = 0 (and the flag) where they make no sense.
__device__ __forceinline__ void seq_info(const Kargs& a, int b, int& r0, int& n, int& T, bool tell) {
  r0 = a.row_start[b];
  const int r1 = a.row_start[b + 1];
  T = a.c.lens[b];
  n = r1 - r0;
  if (r0 < 0 || r1 > a.rows || n < 0 || n > a.max_rows || T < 0 || T > a.c.capacity()) {
    if (tell) flag_error(a.c.status, kErrShape);
    n = 0;
  }
}
// Tiles of one unit of the sequence, and its row tiles of R rows.
__device__ __forceinline__ int unit_tiles(int T) { return (T + kTile - 1) / kTile; }
__device__ __forceinline__ int row_tiles(const Kargs& a, int n, int R) { return (n * a.hpg + R - 1) / R; }

// o / l; a row that sees nothing gives 0, one whose every score is -inf gives NaN (0 / 0), as the formula
__device__ __forceinline__ float finish(float o, float l, int lim) { return lim <= 0 ? 0.f : o / l; }

template <typename KT, bool Q32, int HD, int NB>
__global__ void __launch_bounds__(kThreads) attn_paged_kernel(Kargs a) {
  using S = Shape<KT, Q32, HD, NB>;
  constexpr bool F32 = S::kF32;
  constexpr int R = S::R, MD = HD / 16, kStages = S::kStages;
  constexpr int kCpr = S::kRowBytes / 16;          // 16-byte chunks of a row
  constexpr float kBias = bias_of<KT>();
  using QT = typename std::conditional<Q32, float, KT>::type;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* const stages = smem;
  unsigned char* const qs = stages + kWarps * kStages * S::kStageBytes;
  float* const obuf = reinterpret_cast<float*>(qs + S::kQBytes);
  Desc* const descs = reinterpret_cast<Desc*>(reinterpret_cast<unsigned char*>(obuf) + S::kObufBytes);
  float* const rowc = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(descs) + S::kDescBytes);   // score factor
  int* const slim = reinterpret_cast<int*>(rowc + R);
  float* const mw = reinterpret_cast<float*>(slim + R);       // [kWarps][R]
  float* const lw = mw + kWarps * R;
  float* const mf = lw + kWarps * R;
  float* const lf = mf + R;
  int* const pre = reinterpret_cast<int*>(lf + R);            // [batch + 1]
  __shared__ int wtot[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int B = a.c.batch;
  pdl_wait();
  pdl_trigger();

  int f0, f1, unit_b = 0, unit_kvh = 0, unit_row0 = 0;
  if (a.cluster) {
    // a cluster for each (sequence, kv head, row tile), an equal run of its tiles for each CTA
    const int unit = blockIdx.x / a.cluster, rank = blockIdx.x - unit * a.cluster;
    const int group = unit / a.rb;
    unit_row0 = (unit - group * a.rb) * R;
    unit_b = group / a.c.Hk;
    unit_kvh = group - unit_b * a.c.Hk;
    int r0, n, T;
    seq_info(a, unit_b, r0, n, T, rank == 0 && unit_kvh == 0 && unit_row0 == 0);
    const int per = unit_row0 < n * a.hpg ? unit_tiles(T) : 0, chunk = (per + a.cluster - 1) / a.cluster;
    f0 = min(per, rank * chunk);
    f1 = min(per, f0 + chunk);
    if (tid < R) {   // what a CTA without tiles adds
      mf[tid] = -INFINITY;
      lf[tid] = 0.f;
    }
    if (f0 == f1)
      for (int i = tid; i < R * S::kObufStride; i += kThreads) obuf[i] = 0.f;
  } else {
    // first tile of every sequence
    int carry = 0;
    for (int i0 = 0; i0 < B; i0 += kThreads) {
      const int i = i0 + tid;
      int mine = 0;
      if (i < B) {
        int r0, n, T;
        seq_info(a, i, r0, n, T, blockIdx.x == 0);
        mine = unit_tiles(T) * row_tiles(a, n, R) * a.c.Hk;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += z;
      }
      __syncthreads();
      if (lane == 31) wtot[warp] = incl;
      __syncthreads();
      int base = carry;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += wtot[w];
        carry += wtot[w];
      }
      if (i < B) pre[i + 1] = base + incl;
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int total = pre[B];
    const int chunk = (total + a.grid - 1) / a.grid;
    f0 = min((long long)total, (long long)blockIdx.x * chunk);
    f1 = min(total, f0 + chunk);
    if (f0 == f1) return;
  }
  const int niter = f1 - f0;

  Desc* const my = descs + warp * kRing;
  unsigned char* const mystages = stages + warp * kStages * S::kStageBytes;

  // descriptors of tiles it0 .. it0 + 15, one per lane
  auto look_up = [&](int it0) {
    const int it = it0 + lane, f = f0 + it;
    if (lane < kRing / 2 && it < niter) {
      Desc d;
      int lo = unit_b, tile = f;
      if (!a.cluster) {
        lo = 0;
        int hi = B;                        // the last sequence that begins at or before f
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pre[mid] <= f) lo = mid;
          else hi = mid;
        }
      }
      const int T = a.c.lens[lo], per = unit_tiles(T);
      d.b = lo;
      d.kvh = unit_kvh;
      d.row0 = unit_row0;
      if (!a.cluster) {
        const int rt = row_tiles(a, a.row_start[lo + 1] - a.row_start[lo], R);
        const int rem = f - pre[lo], u = rem / per;
        tile = rem - u * per;
        d.kvh = u / rt;
        d.row0 = (u - d.kvh * rt) * R;
      }
      d.pos0 = tile * kTile + warp * kStep;
      d.ends = (tile == 0 ? 3 : it == 0 ? 1 : 0) | (tile == per - 1 ? 12 : it == niter - 1 ? 4 : 0);
      d.nvalid = max(0, min(kStep, T - d.pos0));
      d.off = -1;
      if (d.nvalid > 0) {
        const int page = a.c.table[(long long)lo * a.c.max_pages + (d.pos0 >> a.c.page_shift)];
        if (page >= 0 && page < a.c.n_pages)
          d.off = page * a.c.page_stride + (((long long)d.kvh << a.c.page_shift) + (d.pos0 & (a.c.page() - 1))) * HD;
        else
          flag_error(a.c.status, kErrShape);
      }
      my[it & (kRing - 1)] = d;
    }
    __syncwarp();
  };
  auto issue = [&](int it) {
    const Desc& d = my[it & (kRing - 1)];
    const int nv = d.nvalid;
    if (nv > 0) {
      const long long off = d.off;
      const uint32_t sk = smem_u32(mystages + (it % kStages) * S::kStageBytes);
      const uint32_t sv = sk + kStep * S::kRowBytes;
      const char* gk = static_cast<const char*>(a.c.k);
      const char* gv = static_cast<const char*>(a.c.v);
      if (off >= 0) {
        gk += off * (long long)sizeof(KT);
        gv += off * (long long)sizeof(KT);
      }
      const int c = lane % kCpr, r0 = lane / kCpr;
      constexpr int kRows = 32 / kCpr;   // rows one pass of the warp copies
      if (off >= 0 && nv == kStep) {
#pragma unroll
        for (int i = 0; i < kStep / kRows; ++i) {
          const int r = i * kRows + r0;
          cp16(sk + r * S::kRowBytes + swz_k<F32>(c, r) * 16, gk + r * S::kRowBytes + c * 16);
          cp16(sv + r * S::kRowBytes + swz_v<F32>(c, r) * 16, gv + r * S::kRowBytes + c * 16);
        }
      } else {
        // what lies behind the sequence's end (or in no page) is read as zero: stale rows may hold anything
#pragma unroll
        for (int i = 0; i < kStep / kRows; ++i) {
          const int r = i * kRows + r0;
          const bool take = off >= 0 && r < nv;
          const int rr = take ? r : 0;
          cp16_or_zero(sk + r * S::kRowBytes + swz_k<F32>(c, r) * 16, gk + rr * S::kRowBytes + (take ? c * 16 : 0), take);
          cp16_or_zero(sv + r * S::kRowBytes + swz_v<F32>(c, r) * 16, gv + rr * S::kRowBytes + (take ? c * 16 : 0), take);
        }
      }
    }
    cp_commit();
  };

  // B fragments of row tile nb's elements 16 ks .. 16 ks + 31, from the hi (0) or the lo plane
  auto load_q = [&](uint32_t (&t)[4], int nb, int ks, int plane) {
    const int r = nb * 8 + (lane & 7), c = 2 * ks + (lane >> 3);
    ldsm4(t, smem_u32(qs) + (plane * R * HD + r * HD + ((c ^ (r & 7)) << 3)) * 2);
  };

  // The transposed fragments of V's elements 16 md .. 16 md + 31 of the staged step.
  auto load_v = [&](uint32_t (&va)[2][4], uint32_t vu, int md) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = (lane & 7) + 8 * (lane >> 4), c = 2 * (md + u) + ((lane >> 3) & 1);
      ldsm4t(va[u], vu + r * S::kRowBytes + swz_v<false>(c, r) * 16);
    }
  };
  // Probabilities as B fragments (positions 2 t4, 2 t4 + 1 (+ 8 i) of row g8), hi and what it leaves
  auto pairs = [&](const float (&p)[NB][4], uint32_t (&ph)[NB][2], uint32_t (&pl)[NB][2]) {
    if constexpr (!F32) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float ra, rb, za, zb;
          const uint32_t h = Two<KT>::pack(p[nb][2 * i], p[nb][2 * i + 1], ra, rb);
          if constexpr (Q32) mul2(ra, rb, kLoUp);
          const uint32_t w = Two<KT>::pack(ra, rb, za, zb);
          ph[nb][i] = transpose8(h);
          pl[nb][i] = transpose8(w);
        }
    }
  };

  // A unit's sequence and query rows (one warp, every fourth row), read before they are needed: ahead of the first
  // copies of K and V, which would hold them up, and for a later unit ahead of the merge of the one before.
  constexpr int kQRows = R / kWarps;
  constexpr bool kEarly = NB <= 2;   // else the registers are full until the merge is done
  float xq[kQRows][HD / 32];
  int next_r0 = 0, next_n = 0, next_T = 0;
  auto fetch_rows = [&](const Desc& e) {
    seq_info(a, e.b, next_r0, next_n, next_T, false);
#pragma unroll
    for (int j = 0; j < kQRows; ++j) {
      const int rr = e.row0 + warp + j * kWarps, i = rr / a.hpg, h = rr - i * a.hpg;
      const QT* src = static_cast<const QT*>(a.q) + (next_r0 + (i < next_n ? i : 0)) * a.ldq + (long long)(e.kvh * a.hpg + h) * HD;
#pragma unroll
      for (int k = 0; k < HD / 32; ++k) xq[j][k] = i < next_n ? as_float<QT>(src[k * 32 + lane]) : 0.f;
    }
  };

  look_up(0);
  if (niter > 0) fetch_rows(my[0]);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < niter) issue(s);
    else cp_commit();
  }

  // Score fragments: positions g8 + 8 (k >> 1) of the step, rows 8 nb + 2 t4 + (k & 1) of the tile; the rows of O's
  // fragments are the same, its elements dim_of(md, k).  m is what the exponents refer to: at most kSlack below the
  // maximum so far.
  auto dim_of = [&](int md, int k) { return F32 ? 32 * (md >> 1) + 4 * g8 + 2 * (md & 1) + (k >> 1) : 16 * md + g8 + 8 * (k >> 1); };
  float m[NB][2], l[NB][2], O[NB][MD][4];
  float fac[NB][2];
  int lim[NB][2];
  uint32_t qreg[S::kQRegs ? NB : 1][S::kQRegs ? MD : 1][Q32 ? 4 : 2];
  int seq_r0 = 0, seq_n = 0, seq_T = 0, least = 0;
  bool begins_unit = false;

  for (int it = 0; it < niter; ++it) {
    {
      // the next copies' tiles, and the one behind this for its unit's rows
      constexpr int kAhead = kStages > 1 ? kStages - 1 : 1;
      if (it + kAhead < niter && ((it + kAhead) & (kRing / 2 - 1)) == 0) look_up(it + kAhead);
      const int nx = it + kStages - 1;
      if (nx < niter) {
        issue(nx);
      } else {
        cp_commit();
      }
    }
    const Desc d = my[it & (kRing - 1)];
    const int kvh = d.kvh, tile_row = d.row0;

    if (d.ends & 1) {
      begins_unit = d.ends & 2;
      __syncthreads();   // the previous unit's rows and sums are no longer read
      seq_r0 = next_r0;
      seq_n = next_n;
      seq_T = next_T;
      least = seq_T - seq_n + 1;   // positions that every row of the sequence sees
#pragma unroll
      for (int j = 0; j < kQRows; ++j) {
        const int r = warp + j * kWarps, i = (tile_row + r) / a.hpg;
        const bool real = i < seq_n;
        const float (&x)[HD / 32] = xq[j];
        float f = a.scale2;
        if constexpr (F32) {
#pragma unroll
          for (int k = 0; k < HD / 32; ++k) {
            const int e = k * 32 + lane;
            reinterpret_cast<float*>(qs)[r * HD + swz_k<true>(e >> 2, r) * 4 + (e & 3)] = x[k];
          }
        } else {
          KT* hi = reinterpret_cast<KT*>(qs);
          float up = 1.f;
          if constexpr (Q32) {
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < HD / 32; ++k) top = fmaxf(top, fabsf(x[k]));
            top = warp_max(top);
            // the row's largest element to [2^13, 2^14): its half keeps 11 bits and its rest 11 more.  Subnormal ones go
            // up by 2^126 (what is left of their bits fits the pair then, too), so that 2^-e stays a normal number.
            if (top > 0.f && top < INFINITY) {
              int e;
              frexpf(top, &e);
              e = min(126, 14 - e);
              up = ldexpf(1.f, e);
              f = a.scale2 * ldexpf(1.f, -e);
            }
          }
#pragma unroll
          for (int k = 0; k < HD / 32; ++k) {
            const int e = k * 32 + lane;
            const int at = r * HD + (((e >> 3) ^ (r & 7)) << 3) + (e & 7);
            const float y = x[k] * up;
            const KT yh = rounded<KT>(y);
            hi[at] = yh;
            if constexpr (Q32) hi[R * HD + at] = rounded<KT>(y - as_float<KT>(yh));
          }
        }
        if (lane == 0) {
          rowc[r] = f;
          slim[r] = real ? seq_T - seq_n + i + 1 : 0;
        }
      }
      __syncthreads();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[nb][k] = -INFINITY;
          l[nb][k] = 0.f;
          fac[nb][k] = rowc[nb * 8 + 2 * t4 + k];
          lim[nb][k] = slim[nb * 8 + 2 * t4 + k];
        }
#pragma unroll
        for (int md = 0; md < MD; ++md)
#pragma unroll
          for (int k = 0; k < 4; ++k) O[nb][md][k] = 0.f;
        if constexpr (S::kQRegs) {
#pragma unroll
          for (int ks = 0; ks < MD; ks += 2) {
            uint32_t t[4];
            load_q(t, nb, ks, 0);
            qreg[nb][ks][0] = t[0], qreg[nb][ks][1] = t[1], qreg[nb][ks + 1][0] = t[2], qreg[nb][ks + 1][1] = t[3];
            if constexpr (Q32) {
              load_q(t, nb, ks, 1);
              qreg[nb][ks][2] = t[0], qreg[nb][ks][3] = t[1], qreg[nb][ks + 1][2] = t[2], qreg[nb][ks + 1][3] = t[3];
            }
          }
        }
      }
    }

    cp_wait<kStages - 1>();
    __syncwarp();

    if (d.nvalid > 0) {
      const unsigned char* kst = mystages + (it % kStages) * S::kStageBytes;
      const unsigned char* vst = kst + kStep * S::kRowBytes;
      const uint32_t ku = smem_u32(kst), vu = smem_u32(vst);
      // lo: the products with a lo half, where the result is stored in fp32.  They are summed apart, since
      // the tensor cores cut an addition's result off: fewer cuts fall on the large sum.
      constexpr bool kApart = F32 || Q32;
      // Few row tiles: a second sum for every other product, so that none waits for the one before it.
      constexpr bool kTwoSums = !F32 && NB <= 2;
      float sc[NB][4], lo[kApart ? NB : 1][4], sd[kTwoSums ? NB : 1][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[nb][k] = 0.f;
          if constexpr (kApart) lo[nb][k] = 0.f;
          if constexpr (kTwoSums) sd[nb][k] = 0.f;
        }

      // S^T = K Q^T
      if constexpr (!F32) {
#pragma unroll
        for (int ks = 0; ks < MD; ks += 2) {
          uint32_t ka[2][4];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = lane & 15, c = 2 * (ks + u) + (lane >> 4);
            ldsm4(ka[u], ku + r * S::kRowBytes + swz_k<false>(c, r) * 16);
          }
          uint32_t t[S::kQRegs ? 1 : NB][4];
          if constexpr (!S::kQRegs) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) load_q(t[nb], nb, ks, 0);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float(&sum)[4] = kTwoSums && u ? sd[kTwoSums ? nb : 0] : sc[nb];
              if constexpr (S::kQRegs) mma16<KT>(sum, ka[u], qreg[nb][ks + u][0], qreg[nb][ks + u][1]);
              else mma16<KT>(sum, ka[u], t[nb][2 * u], t[nb][2 * u + 1]);
            }
          if constexpr (Q32) {
            if constexpr (!S::kQRegs) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) load_q(t[nb], nb, ks, 1);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if constexpr (S::kQRegs) mma16<KT>(lo[nb], ka[u], qreg[nb][ks + u][2], qreg[nb][ks + u][3]);
                else mma16<KT>(lo[nb], ka[u], t[nb][2 * u], t[nb][2 * u + 1]);
              }
          }
        }
      } else {
        // k index t of a step is element 16 j + 4 t (+ 2 in the second), k index t + 4 the one after it
#pragma unroll 2
        for (int j = 0; j < HD / 16; ++j) {
          const float4 k0 = *reinterpret_cast<const float4*>(kst + g8 * S::kRowBytes + swz_k<true>(4 * j + t4, g8) * 16);
          const float4 k1 = *reinterpret_cast<const float4*>(kst + (g8 + 8) * S::kRowBytes + swz_k<true>(4 * j + t4, g8) * 16);
          uint32_t ah[2][4], al[2][4];
          split_tf32(k0.x, ah[0][0], al[0][0]);
          split_tf32(k1.x, ah[0][1], al[0][1]);
          split_tf32(k0.y, ah[0][2], al[0][2]);
          split_tf32(k1.y, ah[0][3], al[0][3]);
          split_tf32(k0.z, ah[1][0], al[1][0]);
          split_tf32(k1.z, ah[1][1], al[1][1]);
          split_tf32(k0.w, ah[1][2], al[1][2]);
          split_tf32(k1.w, ah[1][3], al[1][3]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int r = nb * 8 + g8;
            const float4 q4 = *reinterpret_cast<const float4*>(qs + (r * HD + swz_k<true>(4 * j + t4, r) * 4) * 4);
            uint32_t bh[4], bl[4];
            split_tf32(q4.x, bh[0], bl[0]);
            split_tf32(q4.y, bh[1], bl[1]);
            split_tf32(q4.z, bh[2], bl[2]);
            split_tf32(q4.w, bh[3], bl[3]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              mma8(lo[nb], al[s], bh[2 * s], bh[2 * s + 1]);
              mma8(lo[nb], ah[s], bl[2 * s], bl[2 * s + 1]);
              mma8(sc[nb], ah[s], bh[2 * s], bh[2 * s + 1]);
            }
          }
        }
      }

      // scores in base 2, masks, reference and sum
      const bool masked = d.pos0 + kStep > least;   // some row does not see all 16
      bool passes = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float s = sc[nb][k];
          if constexpr (kTwoSums) s += sd[nb][k];
          if constexpr (kApart) s += lo[nb][k];
          sc[nb][k] = s * fac[nb][k & 1];
        }
      if (masked) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (d.pos0 + g8 + 8 * (k >> 1) >= lim[nb][k & 1]) sc[nb][k] = -INFINITY;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 4; ++k) passes |= sc[nb][k] > m[nb][k & 1] + kSlack;
      if (a.scores) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (lim[nb][k] > 0) {   // a real row; positions behind the end fall into the capacity's last 16
              float* dst = a.scores + (((long long)d.b * a.c.Hk + kvh) * (a.hpg * a.max_rows) + tile_row + nb * 8 + 2 * t4 + k) * a.c.capacity() + d.pos0 + g8;
              dst[0] = sc[nb][k];
              dst[8] = sc[nb][2 + k];
            }
      }
      if (__any_sync(0xffffffffu, passes)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = fmaxf(sc[nb][k], sc[nb][2 + k]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float mn = fmaxf(m[nb][k], top);
            const float c = ex2(m[nb][k] - (mn == -INFINITY ? 0.f : mn));
            m[nb][k] = mn;
            l[nb][k] *= c;
#pragma unroll
            for (int md = 0; md < MD; ++md) {
              O[nb][md][k] *= c;
              O[nb][md][2 + k] *= c;
            }
          }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float from = kBias - (m[nb][k] == -INFINITY ? 0.f : m[nb][k]);
          sc[nb][k] = ex2(sc[nb][k] + from);
          sc[nb][2 + k] = ex2(sc[nb][2 + k] + from);
          l[nb][k] += sc[nb][k] + sc[nb][2 + k];
        }

      // A masked row takes nothing from a position it does not see, but 0 x inf is NaN: where such
      // positions hold a V that is not finite, the step's P V is added element by element.
      bool odd = false;
      if (masked && seq_n > 1) {
        for (int r = max(0, least - d.pos0); r < d.nvalid; ++r)
          for (int e = lane; e < HD; e += 32) {
            const int c = e * (int)sizeof(KT) / 16;
            const float x = staged<KT>(vst + r * S::kRowBytes + swz_v<F32>(c, r) * 16 + e * sizeof(KT) % 16);
            odd |= !(fabsf(x) < INFINITY);
          }
        odd = __any_sync(0xffffffffu, odd);
      }
      // O^T += V^T P^T
      if (odd) {
        for (int r = 0; r < d.nvalid; ++r)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            float p[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) p[k] = __shfl_sync(0xffffffffu, r & 8 ? sc[nb][2 + k] : sc[nb][k], ((r & 7) << 2) | t4);
#pragma unroll
            for (int md = 0; md < MD; ++md)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = dim_of(md, k);
                const int c = e * (int)sizeof(KT) / 16;
                const float x = staged<KT>(vst + r * S::kRowBytes + swz_v<F32>(c, r) * 16 + e * sizeof(KT) % 16);
                if (d.pos0 + r < lim[nb][k & 1]) O[nb][md][k] = fmaf(p[k & 1], x, O[nb][md][k]);
              }
          }
      } else if constexpr (Q32) {
        auto add = [&](const float (&p)[NB][4], const float (&down)[NB][2]) {
          uint32_t ph[NB][2], pl[NB][2];
          pairs(p, ph, pl);
          // two tiles of elements at a time: products that add to one sum stay 2 NB apart
#pragma unroll
          for (int md = 0; md < MD; md += 2) {
            uint32_t va[2][4];
            load_v(va, vu, md);
            float x[2][NB][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[u][nb][k] = 0.f;
                mma16<KT>(x[u][nb], va[u], pl[nb][0], pl[nb][1]);
              }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int k = 0; k < 4; k += 2) mul2(x[u][nb][k], x[u][nb][k + 1], 1.f / kLoUp);
                mma16<KT>(x[u][nb], va[u], ph[nb][0], ph[nb][1]);
              }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int k = 0; k < 4; k += 2)
                  fma2(O[nb][md + u][k], O[nb][md + u][k + 1], x[u][nb][k], x[u][nb][k + 1], down[nb][0], down[nb][1]);
          }
        };
        unsigned smallest = 0xffffffffu;   // the smallest but 0, by its bits (one less, so that 0 comes last)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < 4; ++k) smallest = min(smallest, __float_as_uint(sc[nb][k]) - 1u);
        float down[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) down[nb][0] = down[nb][1] = 1.f;
        if (!__any_sync(0xffffffffu, smallest < __float_as_uint(kPairFrom) - 1u)) {
          add(sc, down);
        } else {
          // Probabilities that a pair does not hold: each row's largest is brought to [2^9, 2^10) by a power of two, what then
          // is in the pair's range is added and taken out, until nothing is left (each pass takes 23 powers of two).
          bool left = true;
#pragma unroll 1
          while (left) {
            float p[NB][4];
            left = false;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float top = fmaxf(sc[nb][k], sc[nb][2 + k]);
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const unsigned e = max(10u, __float_as_uint(top) >> 23 & 255u);   // 2^126 at most; both factors are normal
                const float up = __uint_as_float((263 - e) << 23);
                down[nb][k] = __uint_as_float((e - 9) << 23);
#pragma unroll
                for (int i = k; i < 4; i += 2) {
                  const float y = sc[nb][i] * up;
                  const bool now = !(y < kPairFrom);   // NaN too
                  p[nb][i] = now ? y : 0.f;
                  sc[nb][i] = now ? 0.f : sc[nb][i];
                  left |= sc[nb][i] >= 0x1p-126f;   // ex2 gives no smaller ones, and one would never come into the range
                }
              }
            add(p, down);
            left = __any_sync(0xffffffffu, left);
          }
        }
      } else if constexpr (!F32) {
        uint32_t ph[NB][2], pl[NB][2];
        pairs(sc, ph, pl);
#pragma unroll
        for (int md = 0; md < MD; md += 2) {   // as above
          uint32_t va[2][4];
          load_v(va, vu, md);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16<KT>(O[nb][md + u], va[u], ph[nb][0], ph[nb][1]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16<KT>(O[nb][md + u], va[u], pl[nb][0], pl[nb][1]);
        }
      } else {
        // k index t is position 8 nt + 2 t, t + 4 the one after it
        uint32_t bh[NB][4], bl[NB][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // lane (g8, t4) takes row g8's probability of position 8 (i >> 1) + 2 t4 + (i & 1)
            const int from = (2 * t4 + (i & 1)) * 4 + (g8 >> 1);
            const float even = __shfl_sync(0xffffffffu, sc[nb][i & 2], from), uneven = __shfl_sync(0xffffffffu, sc[nb][(i & 2) + 1], from);
            split_tf32(g8 & 1 ? uneven : even, bh[nb][i], bl[nb][i]);
          }
#pragma unroll
        for (int J = 0; J < HD / 32; ++J) {
          float x[NB][2][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int k = 0; k < 4; ++k) x[nb][u][k] = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int ra = 8 * nt + 2 * t4, rb = ra + 1;
            const float4 y = *reinterpret_cast<const float4*>(vst + ra * S::kRowBytes + swz_v<true>(8 * J + g8, ra) * 16);
            const float4 z = *reinterpret_cast<const float4*>(vst + rb * S::kRowBytes + swz_v<true>(8 * J + g8, rb) * 16);
            const float ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t vh[4], vl[4];
              split_tf32(ys[2 * u], vh[0], vl[0]);
              split_tf32(ys[2 * u + 1], vh[1], vl[1]);
              split_tf32(zs[2 * u], vh[2], vl[2]);
              split_tf32(zs[2 * u + 1], vh[3], vl[3]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma8(x[nb][u], vl, bh[nb][2 * nt], bh[nb][2 * nt + 1]);
                mma8(x[nb][u], vh, bl[nb][2 * nt], bl[nb][2 * nt + 1]);
                mma8(x[nb][u], vh, bh[nb][2 * nt], bh[nb][2 * nt + 1]);
              }
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int k = 0; k < 4; ++k) O[nb][2 * J + u][k] += x[nb][u][k];
        }
      }
    }
    __syncwarp();   // the ring's next copy goes into this stage

    if (d.ends & 4) {
      if (kEarly && it + 1 < niter) fetch_rows(my[(it + 1) & (kRing - 1)]);
      // the four warps' references and sums, then their weighted sums of V, one warp after the other
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float s = l[nb][k];
          s += __shfl_xor_sync(0xffffffffu, s, 4);
          s += __shfl_xor_sync(0xffffffffu, s, 8);
          s += __shfl_xor_sync(0xffffffffu, s, 16);
          if (g8 == 0) {
            mw[warp * R + nb * 8 + 2 * t4 + k] = m[nb][k];
            lw[warp * R + nb * 8 + 2 * t4 + k] = s;
          }
        }
      __syncthreads();
      if (tid < R) {
        float top = mw[tid];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, mw[w * R + tid]);
        const float safe = top == -INFINITY ? 0.f : top;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += lw[w * R + tid] * ex2(mw[w * R + tid] - safe);
        mf[tid] = top;
        lf[tid] = s;
      }
      __syncthreads();
      float scale[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float top = mf[nb * 8 + 2 * t4 + k];
          scale[nb][k] = ex2(m[nb][k] - (top == -INFINITY ? 0.f : top));
        }
      if constexpr (S::kBufs > 1) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int md = 0; md < MD; ++md)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              obuf[(warp * R + nb * 8 + 2 * t4 + (k & 1)) * S::kObufStride + dim_of(md, k)] = O[nb][md][k] * scale[nb][k & 1];
        __syncthreads();
      } else {
#pragma unroll 1
        for (int round = 0; round < kWarps; ++round) {
          if (warp == round) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float* const rows = obuf + (nb * 8 + 2 * t4) * S::kObufStride;
              float was[MD][4];   // all loads of a row tile before its stores
#pragma unroll
              for (int md = 0; md < MD; ++md)
#pragma unroll
                for (int k = 0; k < 4; ++k) was[md][k] = round ? rows[(k & 1) * S::kObufStride + dim_of(md, k)] : 0.f;
#pragma unroll
              for (int md = 0; md < MD; ++md)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  rows[(k & 1) * S::kObufStride + dim_of(md, k)] = fmaf(O[nb][md][k], scale[nb][k & 1], was[md][k]);
            }
          }
          __syncthreads();
        }
      }
      auto merged = [&](int r, int e) {
        float o = obuf[r * S::kObufStride + e];
#pragma unroll
        for (int w = 1; w < S::kBufs; ++w) o += obuf[(w * R + r) * S::kObufStride + e];
        return o;
      };
      const int real = min(R, seq_n * a.hpg - tile_row);
      if (a.cluster) {   // joined below
        if constexpr (S::kBufs > 1)
          for (int i = tid; i < R * HD; i += kThreads) obuf[i / HD * S::kObufStride + i % HD] = merged(i / HD, i % HD);
      } else if (begins_unit && (d.ends & 8)) {
        QT* dst = static_cast<QT*>(a.out);
        for (int i = tid; i < real * HD; i += kThreads) {
          const int r = i / HD, e = i - r * HD;
          const int rr = tile_row + r, row = rr / a.hpg, h = rr - row * a.hpg;
          const float o = merged(r, e);
          dst[(seq_r0 + row) * a.ldo + (long long)(kvh * a.hpg + h) * HD + e] = rounded<QT>(finish(o, lf[r], slim[r]));
        }
        if (a.scores && tid < real)
          a.stats[((long long)d.b * a.c.Hk + kvh) * (a.hpg * a.max_rows) + tile_row + tid] = make_float2(mf[tid], lf[tid]);
      } else {
        const long long slot = (long long)blockIdx.x * 2 + (begins_unit ? 1 : 0);
        for (int i = tid; i < real * HD; i += kThreads) {
          const int r = i / HD, e = i - r * HD;
          a.part[(slot * R + r) * HD + e] = merged(r, e);
        }
        if (tid < real) a.ml[slot * R + tid] = make_float2(mf[tid], lf[tid]);
      }
      if (!kEarly && it + 1 < niter) fetch_rows(my[(it + 1) & (kRing - 1)]);
    }
  }

  if (a.cluster) {
    // The cluster's pieces, over distributed shared memory: o = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c,
    // in the order of the CTAs; each CTA adds and stores its share of the rows.
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    int r0, n, T;
    seq_info(a, unit_b, r0, n, T, false);
    const int real = min(R, n * a.hpg - unit_row0), rank = cluster.block_rank();
    QT* dst = static_cast<QT*>(a.out);
    for (int i = rank * kThreads + tid; i < real * HD; i += a.cluster * kThreads) {
      const int r = i / HD, e = i - r * HD;
      const int rr = unit_row0 + r, row = rr / a.hpg, h = rr - row * a.hpg;
      float m[kMaxCluster], l[kMaxCluster], o[kMaxCluster], top = -INFINITY;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const bool is = c < a.cluster;
        m[c] = is ? *cluster.map_shared_rank(mf + r, c) : -INFINITY;
        l[c] = is ? *cluster.map_shared_rank(lf + r, c) : 0.f;
        o[c] = is ? *cluster.map_shared_rank(obuf + r * S::kObufStride + e, c) : 0.f;
        top = fmaxf(top, m[c]);
      }
      const float safe = top == -INFINITY ? 0.f : top;
      float so = 0.f, sl = 0.f;
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const float f = ex2(m[c] - safe);
        sl = fmaf(f, l[c], sl);
        so = fmaf(f, o[c], so);
      }
      dst[(r0 + row) * a.ldo + (long long)(unit_kvh * a.hpg + h) * HD + e] = rounded<QT>(finish(so, sl, T - n + row + 1));
      if (a.scores && e == 0) a.stats[((long long)unit_b * a.c.Hk + unit_kvh) * (a.hpg * a.max_rows) + rr] = make_float2(top, sl);
    }
    cluster.sync();   // no CTA leaves while another reads its sums
  }
}

// ---------------------------------------------------------------------------------
// What is left after the main kernel.  The first CTAs of a sequence (none after clusters), some for
// each unit, add the pieces of a cut unit in the order of the CTAs, o = sum_c 2^(m_c - M) o_c /
// sum_c 2^(m_c - M) l_c, and write the rows of sequences that hold nothing.  The others, if there are weights, add to
// w[b][g][t] the sum over the newest rows i and the group's heads of 2^(s - M + bias) / L, from the scores that the
// main kernel left; one thread owns a position, so the order of its sum is fixed.  A cut unit's M and L are worked out
// again by each of them: a kernel between for that alone costs more than the few loads.
//
// Latency is all there is to it, so it starts while the main kernel still runs: lengths and row ranges (inputs
// of the main kernel, whose CTAs have all seen the kernels before it end) are read and the tiles counted before the
// wait, and after it every load but those of the cut rows' (M, L) is issued at once.  A CTA that finds
// nothing to do leaves before the wait; CTA 0 stays for it, so that this grid does not end before the main one.
// ---------------------------------------------------------------------------------
constexpr int kFinishThreads = 256, kFinishWarps = kFinishThreads / 32, kStatRows = 64;
constexpr int kWeightTile = 1024;   // positions of a weighing CTA
constexpr int kLeastItems = 16;   // of four elements each that a joining CTA writes, at least

// The pieces of a cut unit: piece k is the second slot of CTA c0 (it begins the unit), or the first slot of CTA c0 + k.
struct Cut {
  int c0, pieces;
  __device__ __forceinline__ long long slot(int k) const { return (long long)(c0 + k) * 2 + (k == 0 ? 1 : 0); }
};
__device__ __forceinline__ Cut find_cut(const Kargs& a, int first, int total, int kvh, int rt, int row_tiles, int per) {
  const int chunk = (total + a.grid - 1) / a.grid, u0 = first + (kvh * row_tiles + rt) * per;
  Cut c;
  c.c0 = u0 / chunk;
  c.pieces = (u0 + per - 1) / chunk - c.c0 + 1;
  return c;
}
// M and L of a row of a cut unit, by one warp
__device__ __forceinline__ float2 cut_row(const Kargs& a, const Cut& c, int R, int r, int lane) {
  constexpr int U = 4;
  float top = -INFINITY, sum = 0.f;   // of this lane's pieces
  for (int k0 = lane; k0 < c.pieces; k0 += 32 * U) {
    float2 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 32 * u;
      v[u] = k < c.pieces ? a.ml[c.slot(k) * R + r] : make_float2(-INFINITY, 0.f);
    }
    float most = top;
#pragma unroll
    for (int u = 0; u < U; ++u) most = fmaxf(most, v[u].x);
    const float safe = most == -INFINITY ? 0.f : most;
    sum *= ex2(top - safe);
#pragma unroll
    for (int u = 0; u < U; ++u) sum = fmaf(v[u].y, ex2(v[u].x - safe), sum);
    top = most;
  }
  const float all = warp_max(top);
  return make_float2(all, warp_sum(sum * ex2(top - (all == -INFINITY ? 0.f : all))));
}

template <typename QT>
__global__ void __launch_bounds__(kFinishThreads) attn_finish_kernel(Kargs a, int R, float* weights, long long ldw, float bias) {
  __shared__ float sM[kStatRows], sL[kStatRows];
  __shared__ float4 red[kFinishThreads];
  __shared__ int counts[2][kFinishWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, hd = a.c.hd, slices = a.slices, joins = a.cluster ? 0 : a.c.Hk * a.rb * slices;
  int r0, n, T;
  seq_info(a, b, r0, n, T, false);
  int first = 0, total = 0;   // tiles before this sequence's, tiles of all
  if (!a.cluster) {
    for (int i = tid; i < a.c.batch; i += kFinishThreads) {
      int ri, ni, Ti;
      seq_info(a, i, ri, ni, Ti, false);
      const int mine = unit_tiles(Ti) * row_tiles(a, ni, R) * a.c.Hk;
      total += mine;
      if (i < b) first += mine;
    }
    first = __reduce_add_sync(0xffffffffu, first);
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) {
      counts[0][warp] = first;
      counts[1][warp] = total;
    }
    __syncthreads();
    first = total = 0;
#pragma unroll
    for (int w = 0; w < kFinishWarps; ++w) {
      first += counts[0][w];
      total += counts[1][w];
    }
  }
  const int per = unit_tiles(T), rts = row_tiles(a, n, R), rows = n * a.hpg;
  auto leave = [&] {
    if (blockIdx.x == 0 && b == 0) pdl_wait();
    pdl_trigger();
  };

  if ((int)blockIdx.x >= joins) {
    const int chunks = (a.c.capacity() + kWeightTile - 1) / kWeightTile, x = blockIdx.x - joins;
    const int g = x / chunks, t0 = (x - g * chunks) * kWeightTile;
    if (t0 >= T || n <= 0) return leave();
    const long long unit = (long long)b * a.c.Hk + g, most = a.hpg * a.max_rows;
    const float* s = a.scores + unit * most * a.c.capacity();
    float* to = weights + unit * ldw;
    constexpr int P = kWeightTile / kFinishThreads, U = 4;   // positions a thread, rows at a time
    int t[P], sees[P];                                       // the first row that sees position t
    float was[P], w[P], v[U][P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      t[p] = t0 + p * kFinishThreads + tid;
      sees[p] = t[p] < T ? max(0, t[p] - (T - n)) * a.hpg : rows;
      w[p] = 0.f;
    }
    pdl_wait();
    pdl_trigger();
    auto load = [&](int q, int q1) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int p = 0; p < P; ++p)
          v[u][p] = q + u >= sees[p] && q + u < q1 ? s[(long long)(q + u) * a.c.capacity() + t[p]] : 0.f;
    };
#pragma unroll
    for (int p = 0; p < P; ++p) was[p] = t[p] < T ? to[t[p]] : 0.f;
    for (int q0 = 0; q0 < rows; q0 += kStatRows) {
      const int q1 = min(rows, q0 + kStatRows);
      load(q0, q1);
      if (q0) __syncthreads();
      for (int q = q0 + warp; q < q1; q += kFinishWarps) {
        const int rt = q / R;
        Cut c{0, 1};
        if (!a.cluster) c = find_cut(a, first, total, g, rt, rts, per);
        const float2 ml = c.pieces == 1 ? a.stats[unit * most + q] : cut_row(a, c, R, q - rt * R, lane);
        if (lane == 0) {
          sM[q - q0] = ml.x - bias;
          sL[q - q0] = 1.f / ml.y;
        }
      }
      __syncthreads();
      for (int q = q0; q < q1; q += U) {
        if (q != q0) load(q, q1);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int p = 0; p < P; ++p)
            if (q + u >= sees[p] && q + u < q1) w[p] = fmaf(ex2(v[u][p] - sM[q + u - q0]), sL[q + u - q0], w[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (t[p] < T) to[t[p]] = was[p] + w[p];
    return;
  }
  const int unit = blockIdx.x / slices;
  const int kvh = unit / a.rb, rt = unit - kvh * a.rb;
  const int row0 = rt * R, real = min(R, rows - row0);
  if (real <= 0) return leave();
  // this CTA's share of the unit's rows, in items of four elements
  const int vecs = hd / 4, share = (real * vecs + slices - 1) / slices, base = (blockIdx.x - unit * slices) * share;
  const int items = min(share, real * vecs - base);
  if (items <= 0) return leave();
  auto out = [&](int r, int e) {
    const int rr = row0 + r, row = rr / a.hpg, h = rr - row * a.hpg;
    return static_cast<QT*>(a.out) + (r0 + row) * a.ldo + (long long)(kvh * a.hpg + h) * hd + e;
  };
  if (T == 0) {
    pdl_wait();   // rows may be read before the main kernel by none of ours, but order their writes all the same
    pdl_trigger();
    for (int i = tid; i < items; i += kFinishThreads)
      for (int k = 0; k < 4; ++k) out((base + i) / vecs, 4 * ((base + i) % vecs))[k] = rounded<QT>(0.f);
    return;
  }
  const Cut cut = find_cut(a, first, total, kvh, rt, rts, per);
  const int pieces = cut.pieces;
  if (pieces == 1) return leave();
  // threads that share an item's pieces, or items a thread
  const int parts = max(1, min(pieces, kFinishThreads / items)), part = parts > 1 ? tid / items : 0;
  int item = parts > 1 ? tid - part * items : tid, r = (base + item) / vecs, e = 4 * (base + item - r * vecs);
  constexpr int U = 4;
  pdl_wait();
  pdl_trigger();
  float4 x[U];
  float m[U];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * parts;
      const bool is = part < parts && item < items && k < pieces;
      x[u] = is ? *reinterpret_cast<const float4*>(a.part + (cut.slot(k) * R + r) * hd + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      m[u] = is ? a.ml[cut.slot(k) * R + r].x : -INFINITY;
    }
  };
  load(part);
  for (int q = base / vecs + warp; q <= (base + items - 1) / vecs; q += kFinishWarps) {
    const float2 ml = cut_row(a, cut, R, q, lane);
    if (lane == 0) {
      sM[q] = ml.x == -INFINITY ? 0.f : ml.x;
      sL[q] = ml.y;
    }
  }
  __syncthreads();
  while (true) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part < parts && item < items) {
      const float M = sM[r];
      for (int k = part; k < pieces; k += U * parts) {
        if (k != part) load(k);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float c = ex2(m[u] - M);
          o.x = fmaf(c, x[u].x, o.x);
          o.y = fmaf(c, x[u].y, o.y);
          o.z = fmaf(c, x[u].z, o.z);
          o.w = fmaf(c, x[u].w, o.w);
        }
      }
    }
    if (parts > 1) {
      red[tid] = o;
      __syncthreads();
      if (part == 0)
        for (int p = 1; p < parts; ++p) {
          const float4 y = red[tid + p * items];
          o.x += y.x;
          o.y += y.y;
          o.z += y.z;
          o.w += y.w;
        }
    }
    if (part == 0 && item < items) {
      const int lim = T - n + (row0 + r) / a.hpg + 1;
      QT* to = out(r, e);
      to[0] = rounded<QT>(finish(o.x, sL[r], lim));
      to[1] = rounded<QT>(finish(o.y, sL[r], lim));
      to[2] = rounded<QT>(finish(o.z, sL[r], lim));
      to[3] = rounded<QT>(finish(o.w, sL[r], lim));
    }
    item += kFinishThreads;
    if (parts > 1 || item >= items) return;
    r = (base + item) / vecs;
    e = 4 * (base + item - r * vecs);
    load(0);
  }
}

// Row tiles that one pass over the cache serves: 4 fill the registers at 128 elements a head (128 sums a thread), fp32 needs
// more beside them.
template <typename KT>
constexpr int kMostTiles = sizeof(KT) == 4 ? 2 : 4;
// f with the number of row tiles as a type
template <typename KT, typename F>
auto with_nb(int nb, F&& f) {
  if constexpr (kMostTiles<KT> > 2) {
    if (nb == 4) return f(std::integral_constant<int, 4>());
    if (nb == 3) return f(std::integral_constant<int, 3>());
  }
  return nb == 2 ? f(std::integral_constant<int, 2>()) : f(std::integral_constant<int, 1>());
}

// CTAs of a kernel that the registers of an SM hold, set with its attributes before the first plan (one architecture, so the
// same on every device).
template <typename KT, bool Q32, int HD, int NB>
std::atomic<int> g_reg_ctas{0};

// Sizes of one call, the same for the workspace and for the launch.
struct Plan {
  int nb, R, hpg, rb, grid, cluster;
  size_t smem, part, ml, stats, scores, bytes;
};

template <typename KT, bool Q32, int HD>
Plan plan_for(const AttnPagedArgs& a, int n_sm) {
  Plan p;
  p.hpg = a.H / a.c.Hk;
  const long long rows = (long long)p.hpg * a.max_rows;
  // rows in tiles of 8, up to kMostTiles a pass over the cache, as even as they go
  const int pass = kMostTiles<KT> * 8;
  p.rb = (int)((rows + pass - 1) / pass);
  p.nb = (int)((rows + p.rb * 8 - 1) / (p.rb * 8));
  p.R = 8 * p.nb;
  p.smem = with_nb<KT>(p.nb, [&](auto nb) { return Shape<KT, Q32, HD, decltype(nb)::value>::smem(a.c.batch); });
  // CTAs an SM: what shared memory and registers leave (28 rows of 64 elements take 254 registers, so that two fit where
  // shared memory would allow three: 45.4 us for 32 sequences of 7 rows and 16 heads, 52.6 planned with three), three at most
  const int regs = with_nb<KT>(p.nb, [](auto nb) { return g_reg_ctas<KT, Q32, HD, decltype(nb)::value>.load(std::memory_order_relaxed); });
  const int fit = std::min((int)((228 * 1024) / (p.smem + 1024)), regs);
  const int per_sm = fit < 1 ? 1 : fit > 3 ? 3 : fit;
  const long long tiles = (long long)a.c.batch * a.c.Hk * p.rb * ((a.c.capacity() + kTile - 1) / kTile);
  const long long resident = (long long)per_sm * n_sm;
  // Few units that are not long: a cluster for each joins its pieces by itself, where all fit the GPU at once.
  const long long units = (long long)a.c.batch * a.c.Hk * p.rb;
  const int unit_most = (a.c.capacity() + kTile - 1) / kTile;
  int C = 1;
  while (C < kMaxCluster && C < unit_most) C *= 2;
  p.cluster = units * C <= resident && unit_most <= kClusterTiles * C ? C : 0;
  p.grid = (int)(p.cluster ? units * C : tiles < resident ? tiles : resident);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  p.part = 0;
  p.ml = p.part + up((size_t)p.grid * 2 * p.R * HD * 4);
  p.stats = p.ml + up((size_t)p.grid * 2 * p.R * 8);
  const size_t most = a.weights ? (size_t)a.c.batch * a.c.Hk * rows : 0;
  p.scores = p.stats + up(most * 8);
  p.bytes = p.scores + up(most * a.c.capacity() * 4);
  return p;
}

template <typename KT, bool Q32, int HD>
cudaError_t attn_go(const Launch& L, const AttnPagedArgs& a, int n_sm, void* ws) {
  using QT = typename std::conditional<Q32, float, KT>::type;
  const Plan p = plan_for<KT, Q32, HD>(a, n_sm);
  char* w = static_cast<char*>(ws);
  Kargs k;
  k.c = a.c;
  k.q = a.q;
  k.out = a.out;
  k.ldq = a.ldq;
  k.ldo = a.ldo;
  k.row_start = a.row_start;
  k.rows = a.rows;
  k.max_rows = a.max_rows;
  k.hpg = p.hpg;
  k.rb = p.rb;
  k.scale2 = a.scale * 1.44269504088896340736f;
  k.part = reinterpret_cast<float*>(w + p.part);
  k.ml = reinterpret_cast<float2*>(w + p.ml);
  k.scores = a.weights ? reinterpret_cast<float*>(w + p.scores) : nullptr;
  k.stats = reinterpret_cast<float2*>(w + p.stats);
  k.grid = p.grid;
  k.cluster = p.cluster;
  cudaError_t e;
  e = with_nb<KT>(p.nb, [&](auto nb) {
    const auto kernel = attn_paged_kernel<KT, Q32, HD, decltype(nb)::value>;
    if (p.cluster) return launch_cluster(L, kernel, p.cluster, dim3(p.grid), dim3(kThreads), p.smem, k);
    return launch_k(L, kernel, dim3(p.grid), dim3(kThreads), p.smem, k);
  });
  // few units: several CTAs join each, so that every load of theirs is under way at once
  k.slices = 1;
  while (k.slices * kLeastItems < p.R * HD / 4 && (long long)a.c.batch * a.c.Hk * p.rb * k.slices < n_sm) k.slices *= 2;
  const int joins = p.cluster ? 0 : a.c.Hk * p.rb * k.slices;
  const int adds = a.weights ? a.c.Hk * ((a.c.capacity() + kWeightTile - 1) / kWeightTile) : 0;
  if (e != cudaSuccess || joins + adds == 0) return e;
  return launch_k(L, attn_finish_kernel<QT>, dim3(joins + adds, a.c.batch), dim3(kFinishThreads), 0, k, p.R, a.weights, a.ldw,
                  bias_of<KT>());
}

// Calls f with the kernel family's template arguments.
template <typename F>
auto with_types(int q_elem, int kv_elem, int hd, F&& f) {
#define MS_CASE(KT, Q32) return hd == 64 ? f.template operator()<KT, Q32, 64>() : f.template operator()<KT, Q32, 128>()
  if (kv_elem == kF32) MS_CASE(float, false);
  if (kv_elem == kBf16) MS_CASE(__nv_bfloat16, false);
  if (q_elem == kF32) MS_CASE(__half, true);
  MS_CASE(__half, false);
#undef MS_CASE
}

struct DoPlan {
  const AttnPagedArgs& a;
  int n_sm;
  template <typename KT, bool Q32, int HD> size_t operator()() { return plan_for<KT, Q32, HD>(a, n_sm).bytes; }
};
struct DoLaunch {
  const Launch& L;
  const AttnPagedArgs& a;
  int n_sm;
  void* ws;
  template <typename KT, bool Q32, int HD> cudaError_t operator()() { return attn_go<KT, Q32, HD>(L, a, n_sm, ws); }
};
struct DoAttrs {
  template <typename KT, bool Q32, int HD> cudaError_t operator()() {
    cudaError_t e = cudaSuccess;
    for (int i = 1; i <= kMostTiles<KT> && e == cudaSuccess; ++i)
      e = with_nb<KT>(i, [&](auto nb) {
        constexpr int NB = decltype(nb)::value;
        int ctas = 0;
        const cudaError_t err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, attn_paged_kernel<KT, Q32, HD, NB>, kThreads, 0);
        if (err != cudaSuccess) return err;
        g_reg_ctas<KT, Q32, HD, NB>.store(ctas, std::memory_order_relaxed);
        return allow_smem(attn_paged_kernel<KT, Q32, HD, NB>, Shape<KT, Q32, HD, NB>::smem(kPagedMaxBatch));
      });
    return e;
  }
};

}  // namespace

size_t attn_paged_workspace(const AttnPagedArgs& a, int q_elem, int n_sm) {
  return with_types(q_elem, a.c.elem, a.c.hd, DoPlan{a, n_sm});
}

cudaError_t launch_attn_paged(const Launch& L, const AttnPagedArgs& a, int q_elem, int n_sm, void* workspace) {
  if (a.rows <= 0) return cudaSuccess;
  return with_types(q_elem, a.c.elem, a.c.hd, DoLaunch{L, a, n_sm, workspace});
}

cudaError_t init_attrs_attn_paged() {
  const int pairs[4][2] = {{kF32, kF32}, {kF32, kElemF16}, {kElemF16, kElemF16}, {kBf16, kBf16}};
  for (auto& p : pairs)
    for (int hd : {64, 128}) {
      const cudaError_t e = with_types(p[0], p[1], hd, DoAttrs{});
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace ms
