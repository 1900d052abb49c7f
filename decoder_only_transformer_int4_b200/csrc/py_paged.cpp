// Python calls of the paged-cache operators, in C++.
//
// A call on the smallest sizes takes 3 to 9 us on the GPU.  Through ctypes its checks, its output
// tensors and the conversion of 15 to 20 arguments took 20 to 28 us of the host; here they take 1 to 2 us
// next to the launches (about 1.7 us each).  The functions check tensors (types, shapes, strides, devices),
// allocate the outputs, make the tensors' device current and call the C entry points on its current stream.
// They return the C status beside the outputs; MsError is raised by the Python side.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <string>

#include "../../include/ms.h"
#include "ms_paged.h"

namespace {

// A ValueError of these words, as a C++ exception that the entry points below turn into Python's.
[[noreturn]] void refuse(const char* name, const std::string& what) {
  C10_THROW_ERROR(ValueError, std::string(name) + ": " + what);
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}
std::string text(const at::Tensor& t) {
  return std::string(c10::toString(t.scalar_type())) + " " + shape_text(t.sizes()) + " on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  return THPVariable_Unpack(o);
}

int elem(const at::Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case at::kFloat: return MS_ELEM_F32;
    case at::kHalf: return MS_ELEM_F16;
    case at::kBFloat16: return MS_ELEM_BF16;
    default: refuse(name, std::string("expected float32, float16 or bfloat16, got ") + c10::toString(t.scalar_type()));
  }
}

// Address of a contiguous tensor of this type, shape and device.
void* flat(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, at::Device dev) {
  if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
    refuse(name, std::string("expected a contiguous ") + c10::toString(type) + " tensor " + shape_text(shape) + " on " + dev.str() + ", got " + text(t));
  return t.data_ptr();
}

// Address and row stride of packed rows [rows, heads, dim]; a row's elements lie together.
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
Rows packed_rows(const at::Tensor& t, const char* name, int64_t heads, int64_t dim, at::ScalarType type, at::Device dev) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != dim || t.scalar_type() != type || t.device() != dev)
    refuse(name, std::string("expected ") + c10::toString(type) + " [rows, " + std::to_string(heads) + ", " + std::to_string(dim) + "] on " + dev.str() +
                     ", got " + text(t));
  if (t.stride(2) != 1 || (t.stride(1) != dim && heads > 1)) refuse(name, "the elements of a row must lie together");
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : heads * dim};
}

// Address and row stride of a float32 matrix with `cols` columns.
Rows matrix(const at::Tensor& t, const char* name, int64_t cols, at::Device dev) {
  if (t.dim() != 2 || t.size(1) != cols || t.scalar_type() != at::kFloat || t.device() != dev || (t.stride(1) != 1 && cols > 1))
    refuse(name, "expected float32 [rows, " + std::to_string(cols) + "] on " + dev.str() + ", got " + text(t));
  return {t.data_ptr(), t.size(0) > 1 ? t.stride(0) : cols};
}

int as_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(name, "out of range");
  return static_cast<int>(v);
}
int int_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return as_int(v, name);
}
float float_arg(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

// A call writes into the tensor: autograd sees a new version of it, so that a backward pass which needs the old values
// is refused by torch instead of reading the new ones.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The cache's description, its device and the tensors that it points into.
struct Kv {
  ms_paged_kv s;
  at::Device dev;
  at::Tensor held[5];
};
constexpr const char* kKvName = "ms_paged_kv";
void free_kv(PyObject* o) { delete static_cast<Kv*>(PyCapsule_GetPointer(o, kKvName)); }
const Kv& kv_arg(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kKvName);
  if (!p) throw python_error();
  return *static_cast<Kv*>(p);
}

void need(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) C10_THROW_ERROR(TypeError, "expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}
bool none(PyObject* o) { return o == Py_None; }

void* current_stream(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

PyObject* give(ms_status s, const at::Tensor* a = nullptr, const at::Tensor* b = nullptr, const at::Tensor* c = nullptr) {
  const at::Tensor* all[3] = {a, b, c};
  int n = 0;
  while (n < 3 && all[n]) ++n;
  THPObjectPtr t(PyTuple_New(1 + n));
  if (!t) throw python_error();
  PyTuple_SET_ITEM(t.get(), 0, PyLong_FromLong(s));
  for (int i = 0; i < n; ++i) PyTuple_SET_ITEM(t.get(), 1 + i, THPVariable_Wrap(*all[i]));
  return t.release();
}

// kv(k, v, table, lens, status or None) -> (handle, kv_heads, head_dim, capacity, batch)
PyObject* py_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 5);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &table = tensor(a[2], "table"), &lens = tensor(a[3], "lens");
  const at::Device dev = k.device();
  if (!dev.is_cuda()) refuse("k", "expected CUDA tensors");
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || v.device() != dev)
    refuse("k and v", "expected the same pages [n_pages, kv_heads, page_size, head_dim]");
  const int64_t np = k.size(0), hk = k.size(1), page = k.size(2), hd = k.size(3);
  // the stride of a dimension of one means nothing
  if (np > 1 && k.stride(0) != v.stride(0)) refuse("k and v", "expected the same stride from page to page");
  for (const at::Tensor* t : {&k, &v})
    if ((t->stride(3) != 1 && hd > 1) || (t->stride(2) != hd && page > 1) || (t->stride(1) != page * hd && hk > 1))
      refuse("k and v", "the elements of a page must lie together");
  if (table.dim() != 2) refuse("table", "expected [batch, max_pages]");
  const int64_t batch = table.size(0), most = table.size(1);
  std::unique_ptr<Kv> kv(new Kv{{}, dev, {k, v, table, lens}});
  kv->s.k = k.data_ptr();
  kv->s.v = v.data_ptr();
  kv->s.elem = elem(k, "k");
  kv->s.n_pages = as_int(np, "k");
  kv->s.page_size = as_int(page, "k");
  kv->s.n_kv_heads = as_int(hk, "k");
  kv->s.head_dim = as_int(hd, "k");
  kv->s.page_stride = np > 1 ? k.stride(0) : hk * page * hd;
  kv->s.table = static_cast<const int32_t*>(flat(table, "table", at::kInt, {batch, most}, dev));
  kv->s.max_pages = as_int(most, "table");
  kv->s.batch = as_int(batch, "table");
  kv->s.lens = static_cast<const int32_t*>(flat(lens, "lens", at::kInt, {batch}, dev));
  kv->s.status = none(a[4]) ? nullptr : static_cast<uint32_t*>(flat(tensor(a[4], "status"), "status", at::kInt, {1}, dev));
  if (!none(a[4])) kv->held[4] = tensor(a[4], "status");
  THPObjectPtr cap(PyCapsule_New(kv.get(), kKvName, free_kv));
  if (!cap) throw python_error();
  kv.release();
  return Py_BuildValue("(OLLLL)", cap.get(), (long long)hk, (long long)hd, (long long)(most * page), (long long)batch);
  END_HANDLE_TH_ERRORS
}

// rope(kv, q or None, k, v, row_start, inv_freq or None, interleaved, mscale, positions or None, out or None)
// -> (status, out or nothing)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 10);
  const Kv& kv = kv_arg(a[0]);
  const int64_t hk = kv.s.n_kv_heads, hd = kv.s.head_dim;
  const at::Tensor &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
  const at::ScalarType type = k.scalar_type();
  const int q_elem = elem(k, "k");
  const Rows kr = packed_rows(k, "k", hk, hd, type, kv.dev), vr = packed_rows(v, "v", hk, hd, type, kv.dev);
  const int64_t rows = k.size(0);
  const c10::OptionalDeviceGuard on(kv.dev);
  Rows qr, orow;
  int64_t heads = 0;
  at::Tensor out;
  if (!none(a[1])) {
    const at::Tensor& q = tensor(a[1], "q");
    heads = q.dim() == 3 ? q.size(1) : 0;
    qr = packed_rows(q, "q", heads, hd, type, kv.dev);
    if (none(a[9])) out = at::empty({rows, heads, hd}, q.options());
    else out = tensor(a[9], "out");
    orow = packed_rows(out, "out", heads, hd, type, kv.dev);
    if (q.size(0) != rows || out.size(0) != rows) refuse("q and out", "expected as many rows as k has");
  } else if (!none(a[9])) {
    refuse("out", "goes with q");
  }
  if (v.size(0) != rows) refuse("v", "expected as many rows as k has");
  const void* start = flat(tensor(a[4], "row_start"), "row_start", at::kInt, {(int64_t)kv.s.batch + 1}, kv.dev);
  int64_t pairs = 0;
  const void* freq = nullptr;
  if (!none(a[5])) {
    const at::Tensor& f = tensor(a[5], "inv_freq");
    pairs = f.dim() == 1 ? f.size(0) : -1;
    freq = flat(f, "inv_freq", at::kDouble, {std::max<int64_t>(pairs, 0)}, kv.dev);
  }
  const int turn = PyObject_IsTrue(a[6]);
  if (turn < 0) throw python_error();
  const float mscale = float_arg(a[7]);
  const void* pos = none(a[8]) ? nullptr : flat(tensor(a[8], "positions"), "positions", at::kInt, {rows}, kv.dev);
  const ms_status s = ms_op_rope_append_paged(&kv.s, qr.p, qr.ld, kr.p, kr.ld, vr.p, vr.ld, q_elem, as_int(rows, "k"), as_int(heads, "q"),
                                              static_cast<const int32_t*>(start), static_cast<const int32_t*>(pos),
                                              static_cast<const double*>(freq), as_int(2 * pairs, "inv_freq"), turn, mscale, orow.p, orow.ld,
                                              current_stream(kv.dev));
  if (s == MS_OK) {
    written(kv.held[0]);
    written(kv.held[1]);
    if (!none(a[9])) written(out);
  }
  return out.defined() ? give(s, &out) : give(s);
  END_HANDLE_TH_ERRORS
}

// attn_workspace(kv, element type, heads, max_rows, weights) -> bytes
PyObject* py_attn_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 5);
  const Kv& kv = kv_arg(a[0]);
  const c10::OptionalDeviceGuard on(kv.dev);
  return PyLong_FromSize_t(ms_op_attn_paged_workspace(&kv.s, int_arg(a[1], "q_dtype"), int_arg(a[2], "heads"), int_arg(a[3], "max_rows"),
                                                      PyObject_IsTrue(a[4]) == 1));
  END_HANDLE_TH_ERRORS
}

// attn(kv, q, row_start, max_rows, scale or None, weights or None, out or None, workspace or None) -> (status, out)
PyObject* py_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 8);
  const Kv& kv = kv_arg(a[0]);
  const int64_t hd = kv.s.head_dim;
  const at::Tensor& q = tensor(a[1], "q");
  const at::ScalarType type = q.scalar_type();
  const int q_elem = elem(q, "q");
  const int64_t heads = q.dim() == 3 ? q.size(1) : 0;
  const Rows qr = packed_rows(q, "q", heads, hd, type, kv.dev);
  const int64_t rows = q.size(0);
  const void* start = flat(tensor(a[2], "row_start"), "row_start", at::kInt, {(int64_t)kv.s.batch + 1}, kv.dev);
  const int max_rows = int_arg(a[3], "max_rows");
  const float scale = none(a[4]) ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(hd))) : float_arg(a[4]);
  float* weights = nullptr;
  int64_t ldw = 0;
  if (!none(a[5])) {
    const at::Tensor& w = tensor(a[5], "weights");
    ldw = w.dim() == 3 ? w.size(2) : 0;
    weights = static_cast<float*>(flat(w, "weights", at::kFloat, {kv.s.batch, kv.s.n_kv_heads, ldw}, kv.dev));
  }
  const c10::OptionalDeviceGuard on(kv.dev);
  // 0 for sizes that the call refuses: nothing is allocated for them
  const size_t bytes = ms_op_attn_paged_workspace(&kv.s, q_elem, as_int(heads, "q"), max_rows, weights != nullptr);
  at::Tensor out, ws;
  if (!none(a[6])) out = tensor(a[6], "out");
  else if (bytes) out = at::empty({rows, heads, hd}, q.options());
  Rows orow;
  if (out.defined()) {
    orow = packed_rows(out, "out", heads, hd, type, kv.dev);
    if (out.size(0) != rows) refuse("q and out", "expected the same number of rows");
  }
  if (!none(a[7])) {
    ws = tensor(a[7], "workspace");
    if (ws.scalar_type() != at::kByte || ws.device() != kv.dev || !ws.is_contiguous()) refuse("workspace", "expected contiguous uint8 on " + kv.dev.str());
  } else if (bytes) {
    ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
  }
  const ms_status s = ms_op_attn_paged(&kv.s, qr.p, qr.ld, q_elem, as_int(rows, "q"), max_rows, as_int(heads, "q"), scale,
                                       static_cast<const int32_t*>(start), orow.p, orow.ld, weights, ldw, ws.defined() ? ws.data_ptr() : nullptr,
                                       ws.defined() ? ws.numel() : 0,
                                       current_stream(kv.dev));
  if (s == MS_OK) {
    if (weights) written(THPVariable_Unpack(a[5]));
    if (!none(a[6])) written(out);
  }
  return out.defined() ? give(s, &out) : give(s);
  END_HANDLE_TH_ERRORS
}

// evict(kv, weights, dst_table, keep, first, recent, weights_out or None) -> (status, kept, weights_out, lens)
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 7);
  const Kv& kv = kv_arg(a[0]);
  const int64_t batch = kv.s.batch, hk = kv.s.n_kv_heads;
  const at::Tensor &w = tensor(a[1], "weights"), &dst = tensor(a[2], "dst_table");
  const int64_t ldw = w.dim() == 3 ? w.size(2) : 0;
  const float* wp = static_cast<const float*>(flat(w, "weights", at::kFloat, {batch, hk, ldw}, kv.dev));
  if (dst.dim() != 2) refuse("dst_table", "expected [batch, pages]");
  const int64_t pages = dst.size(1);
  const void* dp = flat(dst, "dst_table", at::kInt, {batch, pages}, kv.dev);
  const int keep = int_arg(a[3], "keep"), first = int_arg(a[4], "first"), recent = int_arg(a[5], "recent");
  const c10::OptionalDeviceGuard on(kv.dev);
  // refused sizes are found before anything is allocated for them
  const at::Tensor* given = none(a[6]) ? nullptr : &tensor(a[6], "weights_out");
  const int64_t ldwo = !given ? ldw : given->dim() == 3 ? given->size(2) : 0;
  if (given) flat(*given, "weights_out", at::kFloat, {batch, hk, ldwo}, kv.dev);
  const ms_status refused = ms::check_evict_sizes(kv.s, ldw, as_int(pages, "dst_table"), keep, first, recent, ldwo);
  if (refused != MS_OK) return give(refused);
  const at::Tensor wo = given ? *given : at::empty_like(w);
  float* wop = static_cast<float*>(wo.data_ptr());
  const at::Tensor kept = at::empty({batch, hk, keep}, dst.options()), lens = at::empty({batch}, dst.options());
  const ms_status s = ms_op_evict_paged(&kv.s, wp, ldw, static_cast<const int32_t*>(dp), as_int(pages, "dst_table"), keep, first, recent,
                                        static_cast<int32_t*>(kept.data_ptr()), wop, ldwo, static_cast<int32_t*>(lens.data_ptr()),
                                        current_stream(kv.dev));
  if (s == MS_OK) {
    written(kv.held[0]);
    written(kv.held[1]);
    if (given) written(wo);
  }
  return give(s, &kept, &wo, &lens);
  END_HANDLE_TH_ERRORS
}

// verify(target, draft or None, tokens, row_start, max_draft, u_accept, u_sample, status or None) -> (status, accepted, tokens)
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  need(n, 8);
  const at::Tensor &target = tensor(a[0], "target"), &tokens = tensor(a[2], "tokens"), &us = tensor(a[6], "u_sample");
  const at::Device dev = target.device();
  if (!dev.is_cuda()) refuse("target", "expected CUDA tensors");
  if (tokens.dim() != 1 || us.dim() != 1) refuse("tokens and u_sample", "expected one dimension");
  const int64_t rows = tokens.size(0), batch = us.size(0), vocab = target.dim() == 2 ? target.size(1) : 0;
  const Rows t = matrix(target, "target", vocab, dev);
  if (target.size(0) != rows + batch) refuse("target", "expected a row for every draft and one more for every sequence");
  Rows d;
  if (!none(a[1])) {
    const at::Tensor& draft = tensor(a[1], "draft");
    d = matrix(draft, "draft", vocab, dev);
    if (draft.size(0) != rows) refuse("draft", "expected a row for every draft");
    if (rows == 0) d = {};   // no draft, no distribution
  }
  const void* tok = flat(tokens, "tokens", at::kInt, {rows}, dev);
  const void* start = flat(tensor(a[3], "row_start"), "row_start", at::kInt, {batch + 1}, dev);
  const int max_draft = int_arg(a[4], "max_draft");
  const void* ua = flat(tensor(a[5], "u_accept"), "u_accept", at::kFloat, {rows}, dev);
  const void* up = flat(us, "u_sample", at::kFloat, {batch}, dev);
  uint32_t* word = none(a[7]) ? nullptr : static_cast<uint32_t*>(flat(tensor(a[7], "status"), "status", at::kInt, {1}, dev));
  const c10::OptionalDeviceGuard on(dev);
  const at::Tensor accepted = at::empty({batch}, tokens.options()), out = at::empty({batch, (int64_t)std::max(max_draft, 0) + 1}, tokens.options());
  ms_status s = MS_OK;
  if (batch > 0)
    s = ms_op_verify_draft(static_cast<const float*>(t.p), t.ld, static_cast<const float*>(d.p), d.ld, static_cast<const int32_t*>(tok),
                           static_cast<const int32_t*>(start), as_int(rows, "tokens"), as_int(batch, "u_sample"), max_draft, as_int(vocab, "target"),
                           static_cast<const float*>(ua), static_cast<const float*>(up), static_cast<int32_t*>(accepted.data_ptr()),
                           static_cast<int32_t*>(out.data_ptr()), word, current_stream(dev));
  return give(s, &accepted, &out);
  END_HANDLE_TH_ERRORS
}

#define MS_FN(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MS_FN("kv", py_kv),           MS_FN("rope", py_rope),     MS_FN("attn_workspace", py_attn_workspace),
                         MS_FN("attn", py_attn),       MS_FN("evict", py_evict),   MS_FN("verify", py_verify),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__paged(void) { return PyModule_Create(&module); }
