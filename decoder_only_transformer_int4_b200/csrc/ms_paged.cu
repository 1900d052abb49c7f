// C entry points of the paged-cache operators: argument checks, then the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <mutex>

#include "../../include/ms.h"
#include "ms_kernels.h"
#include "ms_paged.h"

namespace {

ms_status bad(ms_status s, const char* who, const char* what) {
  char buf[256];
  snprintf(buf, sizeof(buf), "%s: %s", who, what);
  ms::set_last_error(buf);
  return s;
}
ms_status done(cudaError_t e, const char* who) { return e == cudaSuccess ? MS_OK : bad(MS_ERR_CUDA, who, cudaGetErrorString(e)); }

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
// every int32 or fp32 array among the arguments (null ones are checked apart)
template <typename... Ptr>
bool aligned4(Ptr... p) { return (aligned(p, 4) && ...); }
constexpr int kMostRows = 1 << 30;   // row and block indices are ints, and some are rounded up
size_t elem_bytes(int e) { return e == MS_ELEM_F32 ? 4 : 2; }

// MS_OK, or the reason why the cache cannot be used.
ms_status check_kv(const ms_paged_kv* kv, const char* who) {
  if (!kv) return bad(MS_ERR_INVALID_ARG, who, "null cache");
  if (!kv->k || !kv->v || !kv->table || !kv->lens) return bad(MS_ERR_INVALID_ARG, who, "null pointer in the cache");
  if (kv->elem < MS_ELEM_F32 || kv->elem > MS_ELEM_BF16) return bad(MS_ERR_INVALID_ARG, who, "unknown element type");
  if (kv->page_size < 16 || (kv->page_size & (kv->page_size - 1)) || kv->page_size > (1 << 20))
    return bad(MS_ERR_SHAPE, who, "page_size must be a power of two of at least 16");
  if (kv->head_dim != 64 && kv->head_dim != 128) return bad(MS_ERR_SHAPE, who, "head_dim must be 64 or 128");
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 4096 || kv->n_pages < 1)
    return bad(MS_ERR_SHAPE, who, "need n_pages >= 1 and 1 <= n_kv_heads <= 4096");
  if (kv->batch < 1 || kv->batch > ms::kPagedMaxBatch) return bad(MS_ERR_SHAPE, who, "batch must be in [1, 1024]");
  if (kv->max_pages < 1 || (long long)kv->max_pages * kv->page_size >= (1ll << 30))
    return bad(MS_ERR_SHAPE, who, "need max_pages >= 1 and max_pages * page_size < 2^30");
  const long long page = (long long)kv->n_kv_heads * kv->page_size * kv->head_dim;
  if (kv->page_stride < page || kv->page_stride > (1ll << 40) || kv->page_stride * (long long)elem_bytes(kv->elem) % 16)
    return bad(MS_ERR_SHAPE, who, "page_stride must hold a page and be a multiple of 16 bytes");
  if (!aligned4(kv->table, kv->lens, kv->status)) return bad(MS_ERR_INVALID_ARG, who, "a pointer is not aligned to its elements");
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return bad(MS_ERR_INVALID_ARG, who, "the pages must be 16-byte aligned");
  return MS_OK;
}

ms::PagedView view(const ms_paged_kv& kv) {
  int shift = 0;
  while ((1 << shift) < kv.page_size) ++shift;
  return {kv.k,         kv.v,     kv.elem,      kv.n_pages, shift,   kv.n_kv_heads, kv.head_dim,
          kv.page_stride, kv.table, kv.max_pages, kv.batch,   kv.lens, kv.status};
}

bool types_ok(int q, int kv) {
  return (q == MS_ELEM_F32 && (kv == MS_ELEM_F32 || kv == MS_ELEM_F16)) || (q == kv && (q == MS_ELEM_F16 || q == MS_ELEM_BF16));
}

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];   // SMs of each device whose kernel attributes are set

cudaError_t ready(int* n_sm) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_sms[dev]) {
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = ms::init_attrs_attn_paged();
    if (e != cudaSuccess) return e;
    g_sms[dev] = n > 0 ? n : 1;
  }
  *n_sm = g_sms[dev];
  return cudaSuccess;
}

// Sizes of an attention call; the pointers are checked by the call itself.
ms_status check_attn(const ms_paged_kv* kv, int q_elem, int n_heads, int max_rows, const char* who) {
  const ms_status s = check_kv(kv, who);
  if (s != MS_OK) return s;
  if (!types_ok(q_elem, kv->elem)) return bad(MS_ERR_UNSUPPORTED, who, "this pair of query and cache types is not supported");
  if (n_heads < 1 || n_heads % kv->n_kv_heads || n_heads / kv->n_kv_heads > 256)
    return bad(MS_ERR_SHAPE, who, "n_heads must be a multiple of n_kv_heads, at most 256 times it");
  if (max_rows < 1 || max_rows > 64) return bad(MS_ERR_SHAPE, who, "max_rows must be in [1, 64]");
  const long long tiles = (long long)kv->batch * n_heads * max_rows * (((long long)kv->max_pages * kv->page_size + 63) / 64);
  // the kernel counts in int, and adds a CTA's run to the count
  if (tiles > (1ll << 30)) return bad(MS_ERR_SHAPE, who, "batch * n_heads * max_rows * capacity is too large");
  return MS_OK;
}

ms::AttnPagedArgs attn_args(const ms_paged_kv& kv, int n_heads, int max_rows, float* weights) {
  ms::AttnPagedArgs a{};
  a.c = view(kv);
  a.H = n_heads;
  a.max_rows = max_rows;
  a.weights = weights;
  return a;
}

}  // namespace

namespace ms {

ms_status check_evict_sizes(const ms_paged_kv& kv, int64_t ldw, int dst_pages, int keep, int first, int recent, int64_t ldw_out) {
  const char* who = "ms_op_evict_paged";
  if (keep < 1 || first < 0 || recent < 0 || (int64_t)first + recent > keep)
    return bad(MS_ERR_SHAPE, who, "need keep >= 1, first, recent >= 0 and first + recent <= keep");
  const int64_t capacity = (int64_t)kv.max_pages * kv.page_size;
  if (dst_pages < 1) return bad(MS_ERR_SHAPE, who, "need dst_pages >= 1");
  if (ldw < capacity || ldw_out < (keep < capacity ? keep : capacity) || ldw > (1ll << 40) || ldw_out > (1ll << 40))
    return bad(MS_ERR_SHAPE, who, "need ldw >= max_pages * page_size and ldw_out >= min(keep, max_pages * page_size)");
  return MS_OK;
}

}  // namespace ms

extern "C" {

ms_status ms_op_status(uint32_t* status, void* stream) {
  if (!status || !aligned4(status)) return bad(MS_ERR_INVALID_ARG, "ms_op_status", "null or unaligned status word");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t bits = 0;
  cudaError_t e = cudaMemcpyAsync(&bits, status, sizeof(bits), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(status, 0, sizeof(bits), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return done(e, "ms_op_status");
  if (bits & ms::kErrShapeBit)
    return bad(MS_ERR_SHAPE, "ms_op_status", "a length, row range or page was out of its limits");
  if (bits & ms::kErrTokenBit)
    return bad(MS_ERR_TOKEN_RANGE, "ms_op_status", "a token or random number was out of range, or probabilities summed to nothing");
  return MS_OK;
}

ms_status ms_op_rope_append_paged(const ms_paged_kv* kv, const void* q, int64_t ldq, const void* k, int64_t ldk,
                                  const void* v, int64_t ldv, int q_elem, int rows, int n_heads,
                                  const int32_t* row_start, const int32_t* positions, const double* inv_freq,
                                  int rotary_dim, int interleaved, float mscale, void* q_out, int64_t ldq_out,
                                  void* stream) {
  const char* who = "ms_op_rope_append_paged";
  const ms_status s = check_kv(kv, who);
  if (s != MS_OK) return s;
  if (rows < 0 || rows > kMostRows) return bad(MS_ERR_SHAPE, who, "rows must be in [0, 2^30]");
  if (rows > 0 && (!k || !v)) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (!row_start || (rotary_dim > 0 && !inv_freq)) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (rows > 0 && !q != !q_out) return bad(MS_ERR_INVALID_ARG, who, "q and q_out go together");
  if (!types_ok(q_elem, kv->elem)) return bad(MS_ERR_UNSUPPORTED, who, "this pair of row and cache types is not supported");
  if (rotary_dim < 0 || rotary_dim > kv->head_dim || rotary_dim % 2)
    return bad(MS_ERR_SHAPE, who, "rotary_dim must be even and at most head_dim");
  if (q && (n_heads < 1 || n_heads > (1 << 16))) return bad(MS_ERR_SHAPE, who, "n_heads must be in [1, 65536]");
  const int64_t kw = (int64_t)kv->n_kv_heads * kv->head_dim, qw = (int64_t)n_heads * kv->head_dim;
  const int64_t most = 1ll << 40;
  if (ldk < kw || ldv < kw || (q && (ldq < qw || ldq_out < qw)) || ldk > most || ldv > most || (q && (ldq > most || ldq_out > most)))
    return bad(MS_ERR_SHAPE, who, "a row stride is smaller than its row");
  if (q && q_out == q && ldq_out != ldq && rows > 1) return bad(MS_ERR_SHAPE, who, "in place, ldq_out must be ldq");
  const size_t eb = elem_bytes(q_elem);
  if (!aligned(k, eb) || !aligned(v, eb) || !aligned(q, eb) || !aligned(q_out, eb) || !aligned(inv_freq, 8) || !aligned4(row_start, positions))
    return bad(MS_ERR_INVALID_ARG, who, "a pointer is not aligned to its elements");
  if (rows == 0) return MS_OK;
  int n_sm = 0;
  const cudaError_t e = ready(&n_sm);
  if (e != cudaSuccess) return done(e, who);
  ms::RopeArgs a{view(*kv), q,       k,          v,         ldq,                 ldk,    ldv,      ldq_out,   q_out,
                 rows,      q ? n_heads : 0, rotary_dim, interleaved ? 1 : 0, mscale, inv_freq, row_start, positions};
  const ms::Launch L{static_cast<cudaStream_t>(stream), true, kv->status};
  return done(ms::launch_rope_append_paged(L, a, q_elem, n_sm), who);
}

size_t ms_op_attn_paged_workspace(const ms_paged_kv* kv, int q_elem, int n_heads, int max_rows, int with_weights) {
  const char* who = "ms_op_attn_paged_workspace";
  if (check_attn(kv, q_elem, n_heads, max_rows, who) != MS_OK) return 0;
  int n_sm = 0;
  const cudaError_t e = ready(&n_sm);
  if (e != cudaSuccess) {
    done(e, who);
    return 0;
  }
  float some = 0.f;
  return ms::attn_paged_workspace(attn_args(*kv, n_heads, max_rows, with_weights ? &some : nullptr), q_elem, n_sm);
}

ms_status ms_op_attn_paged(const ms_paged_kv* kv, const void* q, int64_t ldq, int q_elem, int rows, int max_rows,
                           int n_heads, float scale, const int32_t* row_start, void* out, int64_t ldo,
                           float* weights, int64_t ldw, void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "ms_op_attn_paged";
  const ms_status s = check_attn(kv, q_elem, n_heads, max_rows, who);
  if (s != MS_OK) return s;
  if (rows < 0 || rows > kMostRows) return bad(MS_ERR_SHAPE, who, "rows must be in [0, 2^30]");
  if (!row_start || !workspace || (rows > 0 && (!q || !out))) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (!std::isfinite(scale)) return bad(MS_ERR_INVALID_ARG, who, "scale must be finite");
  const int64_t qw = (int64_t)n_heads * kv->head_dim, most = 1ll << 40;
  if (ldq < qw || ldo < qw || ldq > most || ldo > most) return bad(MS_ERR_SHAPE, who, "a row stride is smaller than its row");
  if (q && out == q && ldo != ldq && rows > 1) return bad(MS_ERR_SHAPE, who, "in place, ldo must be ldq");
  if (weights && (ldw < (int64_t)kv->max_pages * kv->page_size || ldw > most))
    return bad(MS_ERR_SHAPE, who, "ldw must hold max_pages * page_size positions");
  const size_t eb = elem_bytes(q_elem);
  if (!aligned(q, eb) || !aligned(out, eb) || !aligned4(weights, row_start))
    return bad(MS_ERR_INVALID_ARG, who, "a pointer is not aligned to its elements");
  if (!aligned(workspace, 256)) return bad(MS_ERR_INVALID_ARG, who, "the workspace must be 256-byte aligned");
  int n_sm = 0;
  const cudaError_t e = ready(&n_sm);
  if (e != cudaSuccess) return done(e, who);
  ms::AttnPagedArgs a = attn_args(*kv, n_heads, max_rows, weights);
  if (workspace_bytes < ms::attn_paged_workspace(a, q_elem, n_sm))
    return bad(MS_ERR_SHAPE, who, "the workspace is too small (ms_op_attn_paged_workspace)");
  a.q = q;
  a.out = out;
  a.ldq = ldq;
  a.ldo = ldo;
  a.row_start = row_start;
  a.rows = rows;
  a.scale = scale;
  a.ldw = ldw;
  const ms::Launch L{static_cast<cudaStream_t>(stream), true, kv->status};
  return done(ms::launch_attn_paged(L, a, q_elem, n_sm, workspace), who);
}

ms_status ms_op_evict_paged(const ms_paged_kv* kv, const float* weights, int64_t ldw, const int32_t* dst_table,
                            int dst_pages, int keep, int first, int recent, int32_t* kept, float* weights_out,
                            int64_t ldw_out, int32_t* lens_out, void* stream) {
  const char* who = "ms_op_evict_paged";
  const ms_status s = check_kv(kv, who);
  if (s != MS_OK) return s;
  if (!weights || !dst_table || !kept || !weights_out || !lens_out) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (!aligned4(weights, dst_table, kept, weights_out, lens_out)) return bad(MS_ERR_INVALID_ARG, who, "a pointer is not aligned to its elements");
  if (lens_out == kv->lens) return bad(MS_ERR_INVALID_ARG, who, "lens_out must not be the cache's lens");
  const ms_status sizes = ms::check_evict_sizes(*kv, ldw, dst_pages, keep, first, recent, ldw_out);
  if (sizes != MS_OK) return sizes;
  if (weights_out == weights && ldw_out != ldw) return bad(MS_ERR_SHAPE, who, "in place, ldw_out must be ldw");
  int n_sm = 0;
  const cudaError_t e = ready(&n_sm);
  if (e != cudaSuccess) return done(e, who);
  ms::EvictArgs a{view(*kv), weights, ldw, dst_table, dst_pages, keep, first, recent, kept, weights_out, ldw_out, lens_out};
  const ms::Launch L{static_cast<cudaStream_t>(stream), true, kv->status};
  return done(ms::launch_evict_paged(L, a, n_sm), who);
}

ms_status ms_op_verify_draft(const float* target, int64_t ld_target, const float* draft, int64_t ld_draft,
                             const int32_t* tokens, const int32_t* row_start, int rows, int batch, int max_draft,
                             int vocab, const float* u_accept, const float* u_sample, int32_t* accepted, int32_t* out,
                             uint32_t* status, void* stream) {
  const char* who = "ms_op_verify_draft";
  if (!target || !row_start || !u_sample || !accepted || !out) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (rows < 0 || rows > kMostRows || batch < 1 || batch > (1 << 20) || vocab < 1 || vocab > (1 << 30) || max_draft < 0 || max_draft > 256)
    return bad(MS_ERR_SHAPE, who, "need rows <= 2^30, 1 <= batch <= 2^20, 1 <= vocab <= 2^30 and 0 <= max_draft <= 256");
  if (rows > 0 && max_draft > 0 && (!tokens || !u_accept)) return bad(MS_ERR_INVALID_ARG, who, "null pointer");
  if (!aligned4(target, draft, tokens, row_start, u_accept, u_sample, accepted, out, status))
    return bad(MS_ERR_INVALID_ARG, who, "a pointer is not aligned to its elements");
  if (ld_target < vocab || (draft && ld_draft < vocab) || ld_target > (1ll << 40) || ld_draft > (1ll << 40))
    return bad(MS_ERR_SHAPE, who, "a row stride is smaller than the vocabulary");
  int n_sm = 0;
  const cudaError_t e = ready(&n_sm);
  if (e != cudaSuccess) return done(e, who);
  ms::VerifyArgs a{target, draft, ld_target, ld_draft, tokens, row_start, rows, batch, max_draft, vocab, u_accept, u_sample, accepted, out};
  const ms::Launch L{static_cast<cudaStream_t>(stream), true, status};
  return done(ms::launch_verify_draft(L, a, n_sm), who);
}

}  // extern "C"
