// Argument marshalling of the softmax-attention operators for Python (attention.py).
//
// A decoding step's calls take a few microseconds on the GPU; checked and marshalled in Python they
// take 10 to 25 on the host.  These functions do the same checks on the tensors directly, allocate the
// outputs that are not given, and call the C ABI (include/kda.h), whose addresses attention.py hands
// over once (init), so that the package loads one library.  Nothing is kept from one call to the next.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "kda.h"

namespace {

struct Functions {
  decltype(&kda_qk_norm_rope) qk_norm_rope;
  decltype(&kda_qk_norm_rope_bwd) qk_norm_rope_bwd;
  decltype(&kda_qk_norm_rope_bwd_workspace_size) bwd_workspace_size;
  decltype(&kda_kv_append) kv_append;
  decltype(&kda_kv_read) kv_read;
  decltype(&kda_attn_decode) attn_decode;
  decltype(&kda_attn_decode_workspace_size) decode_workspace_size;
} g_fn = {};
PyObject* g_error = nullptr;  // KDAError(status, name)

// A wrong argument, raised as ValueError.
struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};  // the Python error is set

[[noreturn]] void bad(const std::string& what) { throw BadArgument(what); }

// The tensor of an argument, null for None.
const at::Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor_or_none(o, name);
  if (!t) bad(std::string(name) + " must be a tensor");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  return v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError{};
  return v;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}
const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

// The device and stream of one call.
class Call {
 public:
  Call(const at::Tensor& t, PyObject* stream) {
    if (!t.is_cuda()) bad("the tensors must be CUDA tensors");
    index_ = t.get_device();
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(index_);
    stream_ = current.stream();
    if (stream != Py_None) {
      const cudaStream_t given = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
      if (PyErr_Occurred()) throw PythonError{};
      if (given != stream_) {
        stream_ = given;
        side_ = true;
      }
    }
    if (c10::cuda::current_device() != index_) guard_.emplace(index_);
  }
  kda_stream_t stream() const { return reinterpret_cast<kda_stream_t>(stream_); }

  // An allocation that belongs to the call's stream.
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    const c10::Device device(c10::kCUDA, index_);
    if (!side_) return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
    c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(stream_, index_));
    return at::Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
  }

  void check(const at::Tensor& t, const char* name, at::ScalarType type) const {
    if (t.scalar_type() != type) bad(std::string(name) + " must be " + type_name(type) + ", got " + type_name(t.scalar_type()));
    if (!t.is_cuda() || t.get_device() != index_) bad(std::string(name) + " must be on cuda:" + std::to_string(index_));
  }
  // The address of a contiguous tensor of the given type, null for null.
  void* at_(const at::Tensor* t, const char* name, at::ScalarType type) const {
    if (!t) return nullptr;
    check(*t, name, type);
    if (!t->is_contiguous()) bad(std::string(name) + " must be contiguous");
    return t->data_ptr();
  }
  void* shaped(const at::Tensor* t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (t && t->sizes() != shape) bad(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t->sizes()));
    return at_(t, name, type);
  }
  // An output: the given tensor, or a new one.
  void* output(const at::Tensor* given, at::Tensor& made, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (given) return shaped(given, name, type, shape);
    made = empty(shape, type);
    return made.data_ptr();
  }
  // The address of an optional workspace (its status word).
  void* status(const at::Tensor* t) const {
    if (t && t->numel() < 256) bad("workspace must have at least 256 bytes");
    return at_(t, "workspace", at::kByte);
  }

 private:
  int index_ = 0;
  cudaStream_t stream_ = nullptr;
  bool side_ = false;
  std::optional<c10::cuda::CUDAGuard> guard_;
};

// A bf16 tensor [..., heads, D] whose heads are contiguous and whose tokens lie one stride apart.
struct Rows {
  const void* p = nullptr;
  int64_t stride = 0, tokens = 0, heads = 0, d = 0;
};
Rows rows_of(const Call& c, const at::Tensor& t, const char* name) {
  c.check(t, name, at::kBFloat16);
  const at::IntArrayRef shape = t.sizes(), step = t.strides();
  const size_t n = shape.size();
  if (n < 3) bad(std::string(name) + " must be [..., heads, D]");
  Rows r;
  r.p = t.data_ptr();
  r.heads = shape[n - 2];
  r.d = shape[n - 1];
  r.tokens = 1;
  for (size_t i = 0; i + 2 < n; ++i) r.tokens *= shape[i];
  r.stride = r.heads * r.d;
  if (r.tokens * r.heads * r.d == 0) return r;
  if ((r.d > 1 && step[n - 1] != 1) || (r.heads > 1 && step[n - 2] != r.d)) bad(std::string(name) + ": the heads of a token must be contiguous");
  int64_t token = 0, span = 1;  // the step between tokens; dimensions of size one have none
  for (size_t i = n - 2; i-- > 0;) {
    if (shape[i] == 1) continue;
    if (span == 1) token = step[i];
    else if (step[i] != token * span) bad(std::string(name) + ": the tokens must lie one stride apart");
    span *= shape[i];
  }
  if (span > 1) r.stride = token;
  return r;
}

// Queries and keys of the same tokens, either of which may be left out.
struct QK {
  Rows q, k;
  int64_t tokens, d;
};
QK qk_of(const Call& c, const at::Tensor* q, const at::Tensor* k) {
  QK r;
  if (q) r.q = rows_of(c, *q, "q");
  if (k) r.k = rows_of(c, *k, "k");
  if (q && k && (r.q.tokens != r.k.tokens || r.q.d != r.k.d)) bad("q and k must have the same tokens and head size");
  r.tokens = q ? r.q.tokens : r.k.tokens;
  r.d = q ? r.q.d : r.k.d;
  return r;
}

struct Cache {
  void *k, *v;
  float *ks, *vs;
  int64_t pages, heads, page, d, k_step, v_step;
};
Cache cache_of(const Call& c, const at::Tensor& k, const at::Tensor& v, const at::Tensor* ks, const at::Tensor* vs) {
  if ((ks == nullptr) != (vs == nullptr)) bad("k_scale and v_scale go together");
  const at::ScalarType type = ks ? at::kFloat8_e4m3fn : at::kBFloat16;
  if (k.dim() != 4 || v.sizes() != k.sizes()) bad("k_cache and v_cache must be [num_pages, num_kv_heads, page_size, D], both alike");
  Cache r;
  r.pages = k.size(0);
  r.heads = k.size(1);
  r.page = k.size(2);
  r.d = k.size(3);
  const at::Tensor* both[2] = {&k, &v};
  const char* names[2] = {"k_cache", "v_cache"};
  int64_t steps[2];
  for (int i = 0; i < 2; ++i) {
    const at::Tensor& t = *both[i];
    if (t.scalar_type() != type)
      bad(std::string(names[i]) + " must be " + type_name(type) + (ks ? " with" : " without") + " scales, got " + type_name(t.scalar_type()));
    c.check(t, names[i], type);
    if (!t.is_contiguous() &&
        (t.stride(3) != 1 || (r.page > 1 && t.stride(2) != r.d) || (r.heads > 1 && t.stride(1) != r.page * r.d)))
      bad(std::string("the pages of ") + names[i] + " must be contiguous");
    steps[i] = r.pages > 1 ? t.stride(0) : r.heads * r.page * r.d;
  }
  r.k = k.data_ptr();
  r.v = v.data_ptr();
  r.k_step = steps[0];
  r.v_step = steps[1];
  const int64_t lines[3] = {r.pages, r.heads, r.page};
  r.ks = static_cast<float*>(c.shaped(ks, "k_scale", at::kFloat, lines));
  r.vs = static_cast<float*>(c.shaped(vs, "v_scale", at::kFloat, lines));
  return r;
}

struct Rotation {
  const float* table = nullptr;
  const int32_t* positions = nullptr;
  int64_t rot = 0, most = 0;
};
Rotation rotation_of(const Call& c, const at::Tensor* table, const at::Tensor* positions, int64_t tokens) {
  Rotation r;
  if (!table) return r;
  if (table->dim() != 2) bad("cos_sin must be [max_positions, rot_dim]");
  if (!positions) bad("positions are needed with cos_sin");
  if (positions->numel() != tokens) bad("positions must have " + std::to_string(tokens) + " entries, got " + std::to_string(positions->numel()));
  r.table = static_cast<const float*>(c.at_(table, "cos_sin", at::kFloat));
  r.positions = static_cast<const int32_t*>(c.at_(positions, "positions", at::kInt));
  r.rot = table->size(1);
  r.most = table->size(0);
  return r;
}

// Sizes the C ABI takes as 32-bit integers.
int32_t i32(int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) bad("a size is out of range");
  return static_cast<int32_t>(v);
}

void raise_if(kda_status_t st, const char* name) {
  if (st == KDA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), name);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PythonError{};
}

// A new reference to what an output argument became.
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

// qk_norm_rope(q, k, q_weight, k_weight, eps, cos_sin, positions, interleaved, q_out, k_out, workspace, stream)
PyObject* qk_norm_rope(PyObject* const* a) {
  const at::Tensor *q = tensor_or_none(a[0], "q"), *k = tensor_or_none(a[1], "k");
  if (!q && !k) bad("one of q and k must be given");
  Call c(q ? *q : *k, a[11]);
  const QK x = qk_of(c, q, k);
  const Rotation r = rotation_of(c, tensor_or_none(a[5], "cos_sin"), tensor_or_none(a[6], "positions"), x.tokens);
  const int64_t channels[1] = {x.d};
  const float* wq = static_cast<const float*>(c.shaped(tensor_or_none(a[2], "q_weight"), "q_weight", at::kFloat, channels));
  const float* wk = static_cast<const float*>(c.shaped(tensor_or_none(a[3], "k_weight"), "k_weight", at::kFloat, channels));
  at::Tensor q_new, k_new;
  void* qo = q ? c.output(tensor_or_none(a[8], "q_out"), q_new, "q_out", at::kBFloat16, q->sizes()) : nullptr;
  void* ko = k ? c.output(tensor_or_none(a[9], "k_out"), k_new, "k_out", at::kBFloat16, k->sizes()) : nullptr;
  raise_if(g_fn.qk_norm_rope(x.q.p, x.k.p, x.q.stride, x.k.stride, wq, wk, static_cast<float>(number(a[4])), r.table, r.positions,
                             qo, ko, x.tokens, i32(x.q.heads), i32(x.k.heads), i32(x.d), i32(r.rot), i32(r.most), truth(a[7]),
                             c.status(tensor_or_none(a[10], "workspace")), c.stream()),
           "kda_qk_norm_rope");
  return Py_BuildValue("(NN)", q ? result(a[8], q_new) : none(), k ? result(a[9], k_new) : none());
}

// qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight, k_weight, eps, cos_sin, positions, interleaved, workspace, stream)
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
  const at::Tensor *q = tensor_or_none(a[2], "q"), *k = tensor_or_none(a[3], "k");
  const at::Tensor *gq = tensor_or_none(a[0], "d_q_out"), *gk = tensor_or_none(a[1], "d_k_out");
  if (!q && !k) bad("one of q and k must be given");
  if ((gq == nullptr) != (q == nullptr) || (gk == nullptr) != (k == nullptr)) bad("a gradient goes with each of q and k");
  Call c(q ? *q : *k, a[11]);
  const QK x = qk_of(c, q, k);
  const Rotation r = rotation_of(c, tensor_or_none(a[7], "cos_sin"), tensor_or_none(a[8], "positions"), x.tokens);
  const int64_t channels[1] = {x.d};
  const float* wq = static_cast<const float*>(c.shaped(tensor_or_none(a[4], "q_weight"), "q_weight", at::kFloat, channels));
  const float* wk = static_cast<const float*>(c.shaped(tensor_or_none(a[5], "k_weight"), "k_weight", at::kFloat, channels));
  const void* dyq = q ? c.shaped(gq, "d_q_out", at::kBFloat16, q->sizes()) : nullptr;
  const void* dyk = k ? c.shaped(gk, "d_k_out", at::kBFloat16, k->sizes()) : nullptr;
  const at::Tensor* ws = tensor_or_none(a[10], "workspace");
  at::Tensor ws_new, dq, dk, dwq, dwk;
  const int64_t need[1] = {static_cast<int64_t>(g_fn.bwd_workspace_size())};
  if (!ws) ws = &(ws_new = c.empty(need, at::kByte));
  void* wsp = c.at_(ws, "workspace", at::kByte);
  if (q) dq = c.empty(q->sizes(), at::kBFloat16);
  if (k) dk = c.empty(k->sizes(), at::kBFloat16);
  if (wq) dwq = c.empty(channels, at::kFloat);
  if (wk) dwk = c.empty(channels, at::kFloat);
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  raise_if(g_fn.qk_norm_rope_bwd(dyq, dyk, x.q.p, x.k.p, x.q.stride, x.k.stride, wq, wk, static_cast<float>(number(a[6])), r.table,
                                 r.positions, ptr(dq), ptr(dk), static_cast<float*>(ptr(dwq)), static_cast<float*>(ptr(dwk)), x.tokens,
                                 i32(x.q.heads), i32(x.k.heads), i32(x.d), i32(r.rot), i32(r.most), truth(a[9]), wsp,
                                 static_cast<size_t>(ws->numel()), c.stream()),
           "kda_qk_norm_rope_bwd");
  auto out = [](const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : none(); };
  return Py_BuildValue("{s:N,s:N,s:N,s:N}", "dq", out(dq), "dk", out(dk), "dq_weight", out(dwq), "dk_weight", out(dwk));
}

// kv_append(k, v, k_cache, v_cache, slots, k_scale, v_scale, q, q_out, q_weight, k_weight, eps, cos_sin, positions, interleaved,
//           workspace, stream)
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[4], "slots");
  const at::Tensor* q = tensor_or_none(a[7], "q");
  Call c(k, a[16]);
  const Cache s = cache_of(c, tensor(a[2], "k_cache"), tensor(a[3], "v_cache"), tensor_or_none(a[5], "k_scale"), tensor_or_none(a[6], "v_scale"));
  const QK x = qk_of(c, q, &k);
  const Rows vr = rows_of(c, v, "v");
  if (x.k.heads != s.heads || x.d != s.d || vr.tokens != x.tokens || vr.heads != s.heads || vr.d != s.d)
    bad("k and v must have the cache's heads and head size, and the same tokens");
  if (slots.numel() != x.tokens) bad("slots must have " + std::to_string(x.tokens) + " entries, got " + std::to_string(slots.numel()));
  const int32_t* sl = static_cast<const int32_t*>(c.at_(&slots, "slots", at::kInt));
  const Rotation r = rotation_of(c, tensor_or_none(a[12], "cos_sin"), tensor_or_none(a[13], "positions"), x.tokens);
  const int64_t channels[1] = {x.d};
  const float* wq = static_cast<const float*>(c.shaped(tensor_or_none(a[9], "q_weight"), "q_weight", at::kFloat, channels));
  const float* wk = static_cast<const float*>(c.shaped(tensor_or_none(a[10], "k_weight"), "k_weight", at::kFloat, channels));
  at::Tensor q_new;
  void* qo = q ? c.output(tensor_or_none(a[8], "q_out"), q_new, "q_out", at::kBFloat16, q->sizes()) : nullptr;
  raise_if(g_fn.kv_append(x.q.p, x.k.p, vr.p, x.q.stride, x.k.stride, vr.stride, wq, wk, static_cast<float>(number(a[11])), r.table,
                          r.positions, qo, s.k, s.v, s.ks, s.vs, sl, x.tokens, i32(x.q.heads), i32(s.heads), i32(s.d), i32(r.rot),
                          i32(r.most), truth(a[14]), i32(s.pages), i32(s.page), s.k_step, s.v_step,
                          c.status(tensor_or_none(a[15], "workspace")), c.stream()),
           "kda_kv_append");
  return q ? result(a[8], q_new) : none();
}

// kv_read(k_cache, v_cache, page_table, cu_seqlens, k_out, v_out, k_scale, v_scale, workspace, stream)
PyObject* kv_read(PyObject* const* a) {
  const at::Tensor &kc = tensor(a[0], "k_cache"), &table = tensor(a[2], "page_table"), &cu = tensor(a[3], "cu_seqlens");
  const at::Tensor &ko = tensor(a[4], "k_out"), &vo = tensor(a[5], "v_out");
  Call c(kc, a[9]);
  const Cache s = cache_of(c, kc, tensor(a[1], "v_cache"), tensor_or_none(a[6], "k_scale"), tensor_or_none(a[7], "v_scale"));
  if (table.dim() != 2 || cu.numel() != table.size(0) + 1) bad("page_table must be [N, max_pages] and cu_seqlens [N + 1]");
  if (ko.dim() != 3 || ko.size(1) != s.heads || ko.size(2) != s.d) bad("k_out must be [total, num_kv_heads, D] of the cache");
  raise_if(g_fn.kv_read(s.k, s.v, s.ks, s.vs, static_cast<const int32_t*>(c.at_(&table, "page_table", at::kInt)),
                        static_cast<const int32_t*>(c.at_(&cu, "cu_seqlens", at::kInt)), c.at_(&ko, "k_out", at::kBFloat16),
                        c.shaped(&vo, "v_out", at::kBFloat16, ko.sizes()), i32(table.size(0)), ko.size(0), i32(s.heads), i32(s.d),
                        i32(s.pages), i32(s.page), i32(table.size(1)), s.k_step, s.v_step,
                        c.status(tensor_or_none(a[8], "workspace")), c.stream()),
           "kda_kv_read");
  Py_INCREF(a[4]);
  Py_INCREF(a[5]);
  return Py_BuildValue("(NN)", a[4], a[5]);
}

// attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, out, lse, k_scale, v_scale, softcap, window, workspace, stream)
PyObject* attn_decode(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "page_table"), &lens = tensor(a[4], "seq_lens");
  Call c(q, a[13]);
  const Cache s = cache_of(c, tensor(a[1], "k_cache"), tensor(a[2], "v_cache"), tensor_or_none(a[8], "k_scale"), tensor_or_none(a[9], "v_scale"));
  const at::IntArrayRef shape = q.sizes();
  const size_t n = shape.size();
  if (n != 3 && n != 4) bad("q must be [B, T, Hq, D] or [B, Hq, D]");
  const int64_t b = shape[0], fresh = n == 4 ? shape[1] : 1, hq = shape[n - 2];
  if (shape[n - 1] != s.d) bad("q must have the cache's head size");
  if (table.dim() != 2 || table.size(0) != b) bad("page_table must be [B, max_pages]");
  const void* qp = c.at_(&q, "q", at::kBFloat16);
  const int32_t* pt = static_cast<const int32_t*>(c.at_(&table, "page_table", at::kInt));
  const int64_t batch[1] = {b};
  const int32_t* sl = static_cast<const int32_t*>(c.shaped(&lens, "seq_lens", at::kInt, batch));
  at::Tensor out_new, ws_new;
  void* op = c.output(tensor_or_none(a[6], "out"), out_new, "out", at::kBFloat16, shape);
  float* lp = static_cast<float*>(c.shaped(tensor_or_none(a[7], "lse"), "lse", at::kFloat, shape.slice(0, n - 1)));
  const at::Tensor* ws = tensor_or_none(a[12], "workspace");
  const int64_t need[1] = {static_cast<int64_t>(g_fn.decode_workspace_size(i32(fresh), i32(hq), i32(s.heads), i32(s.d)))};
  if (!ws) ws = &(ws_new = c.empty(need, at::kByte));
  void* wsp = c.at_(ws, "workspace", at::kByte);
  raise_if(g_fn.attn_decode(qp, s.k, s.v, s.ks, s.vs, pt, sl, static_cast<float>(number(a[5])), static_cast<float>(number(a[10])),
                            i32(integer(a[11])), op, lp, i32(b), i32(fresh), i32(hq), i32(s.heads), i32(s.d), i32(s.pages), i32(s.page),
                            i32(table.size(1)), s.k_step, s.v_step, wsp, static_cast<size_t>(ws->numel()), c.stream()),
           "kda_attn_decode");
  return result(a[6], out_new);
}

// The Python entry of one function: the number of arguments, and every C++ exception as a Python one.
template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs || !g_error) {
    PyErr_SetString(PyExc_TypeError, g_error ? "wrong number of arguments" : "init has not been called");
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const PythonError&) {
  } catch (const BadArgument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (python_error& e) {
    e.restore();
  } catch (const c10::OutOfMemoryError& e) {
    // torch's own class, as its allocations raise it
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// init(KDAError, address, ...): the error class and the addresses of the C ABI in the order of Functions.
PyObject* init(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "init takes the error class and seven addresses");
    return nullptr;
  }
  void* at[7];
  for (int i = 0; i < 7; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_fn.qk_norm_rope = reinterpret_cast<decltype(g_fn.qk_norm_rope)>(at[0]);
  g_fn.qk_norm_rope_bwd = reinterpret_cast<decltype(g_fn.qk_norm_rope_bwd)>(at[1]);
  g_fn.bwd_workspace_size = reinterpret_cast<decltype(g_fn.bwd_workspace_size)>(at[2]);
  g_fn.kv_append = reinterpret_cast<decltype(g_fn.kv_append)>(at[3]);
  g_fn.kv_read = reinterpret_cast<decltype(g_fn.kv_read)>(at[4]);
  g_fn.attn_decode = reinterpret_cast<decltype(g_fn.attn_decode)>(at[5]);
  g_fn.decode_workspace_size = reinterpret_cast<decltype(g_fn.decode_workspace_size)>(at[6]);
  Py_INCREF(args[0]);
  Py_XDECREF(g_error);
  g_error = args[0];
  return none();
}

template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn, kArgs>));
}

PyMethodDef g_methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", fast<qk_norm_rope, 12>(), METH_FASTCALL, nullptr},
    {"qk_norm_rope_bwd", fast<qk_norm_rope_bwd, 12>(), METH_FASTCALL, nullptr},
    {"kv_append", fast<kv_append, 17>(), METH_FASTCALL, nullptr},
    {"kv_read", fast<kv_read, 10>(), METH_FASTCALL, nullptr},
    {"attn_decode", fast<attn_decode, 14>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() { return PyModule_Create(&g_module); }
