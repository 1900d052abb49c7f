// Internal view of a paged KV cache and the launchers of the operators on it.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include "../../include/ms.h"
#include "ms_kernels.h"

namespace ms {

enum Elem { kF32 = 0, kElemF16 = 1, kBf16 = 2 };

constexpr int kPagedMaxBatch = 1024;   // sequences of one call (their tile counts are scanned in shared memory)

// K and V pages [n_pages][Hk][page][hd] (pages page_stride elements apart); table [batch][max_pages]
// names the page of positions page * j .. of a sequence, lens [batch] its positions.
struct PagedView {
  void* k;
  void* v;
  int elem;                // Elem
  int n_pages, page_shift, Hk, hd;
  long long page_stride;
  const int* table;
  int max_pages, batch;
  const int* lens;
  unsigned* status;        // may be null
  __host__ __device__ int page() const { return 1 << page_shift; }
  __host__ __device__ int capacity() const { return max_pages << page_shift; }
};

struct RopeArgs {
  PagedView c;
  const void *q, *k, *v;   // rows at strides ldq, ldk, ldv (elements); q may be null
  long long ldq, ldk, ldv, ldo;
  void* q_out;
  int rows, H, rot;
  int interleaved;
  float mscale;
  const double* inv_freq;  // [rot / 2]
  const int* row_start;    // [batch + 1]
  const int* positions;    // [rows] or null
};
// (n_sm: the device's SMs, by which all of these lay out their grids)
cudaError_t launch_rope_append_paged(const Launch& L, const RopeArgs& a, int q_elem, int n_sm);

struct AttnPagedArgs {
  PagedView c;
  const void* q;
  void* out;
  long long ldq, ldo;
  const int* row_start;
  int rows, max_rows, H;
  float scale;
  float* weights;          // [batch][Hk][ldw] or null
  long long ldw;
};
// Bytes of workspace for a call of these sizes (the same on every device of one kind).
size_t attn_paged_workspace(const AttnPagedArgs& a, int q_elem, int n_sm);
cudaError_t launch_attn_paged(const Launch& L, const AttnPagedArgs& a, int q_elem, int n_sm, void* workspace);
cudaError_t init_attrs_attn_paged();

struct EvictArgs {
  PagedView c;
  const float* weights;    // [batch][Hk][ldw]
  long long ldw;
  const int* dst_table;    // [batch][dst_pages]
  int dst_pages, keep, first, recent;
  int* kept;               // [batch][Hk][keep]
  float* weights_out;      // [batch][Hk][ldwo]; may be `weights` itself
  long long ldwo;
  int* lens_out;           // [batch]
};
cudaError_t launch_evict_paged(const Launch& L, const EvictArgs& a, int n_sm);
// What ms_op_evict_paged says to these sizes; for callers that allocate the outputs.
ms_status check_evict_sizes(const ms_paged_kv& kv, int64_t ldw, int dst_pages, int keep, int first, int recent, int64_t ldw_out);

struct VerifyArgs {
  const float* target;     // rows at stride ldt
  const float* draft;      // rows at stride ldd, or null: the drafts were certain
  long long ldt, ldd;
  const int* tokens;
  const int* row_start;    // [batch + 1]
  int rows, batch, max_draft, V;
  const float* u_accept;
  const float* u_sample;
  int* accepted;
  int* out;                // [batch][max_draft + 1]
};
cudaError_t launch_verify_draft(const Launch& L, const VerifyArgs& a, int n_sm);

}  // namespace ms
