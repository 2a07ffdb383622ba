// binding.cpp -- the argument checks of seq.py for the ordinary call, in C++: a decode call takes the GPU 5 us, and reading
// some twelve tensors' types, shapes, strides and devices from Python 7 more.  Each function either does the whole call
// (returns out, or the status that the C ABI refused it with), or returns None and has touched nothing: the caller's checks in
// Python then say what is wrong, or serve what is rare (an output to be made, tensor subclasses).
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/tq.h"

namespace {

PyObject* g_stream;  // torch._C._cuda_getCurrentRawStream

struct Args {
  PyObject* const* v;
  Py_ssize_t n;
  c10::Device dev{c10::DeviceType::CPU};
  bool ok = true;

  const at::Tensor* tensor(int i) {
    if (i >= n || !THPVariable_CheckExact(v[i])) return fail();
    const at::Tensor* t = &THPVariable_Unpack(v[i]);
    return t->layout() == at::kStrided ? t : fail();
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  bool none(int i) const { return v[i] == Py_None; }

  // contiguous, of this type, shape and device
  void* full(int i, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || t->sizes() != shape || t->device() != dev || !t->is_contiguous()) return fail(), nullptr;
    return t->data_ptr();
  }
  void* some(int i, at::ScalarType type, at::IntArrayRef shape) { return none(i) ? nullptr : full(i, type, shape); }

  // [tokens, heads, dim], the last dimension contiguous
  const void* heads(int i, at::ScalarType type, at::IntArrayRef* shape, int64_t* token, int64_t* head) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != 3 || t->scalar_type() != type || t->device() != dev) return fail(), nullptr;
    *shape = t->sizes();
    const auto s = t->strides();
    if (s[2] != 1 && (*shape)[2] > 1) return fail(), nullptr;
    *token = (*shape)[0] > 1 ? s[0] : 0;
    *head = (*shape)[1] > 1 ? s[1] : 0;
    return t->data_ptr();
  }

  int64_t integer(int i) {
    const long long x = PyLong_Check(v[i]) ? PyLong_AsLongLong(v[i]) : (ok = false, 0);
    if (x == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return x;
  }
  int32_t integer32(int i) {
    const int64_t x = integer(i);
    if (x != (int32_t)x) ok = false;
    return (int32_t)x;
  }
  float real(int i, double missing = 0) {
    if (missing != 0 && none(i)) return (float)missing;
    if (!PyFloat_Check(v[i]) && !PyLong_Check(v[i])) return ok = false, 0.f;
    const double x = PyFloat_AsDouble(v[i]);
    if (x == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
    return (float)x;
  }
  // a workspace of at least `need` bytes
  void* workspace(int i, int64_t need, int64_t* bytes) {
    *bytes = 0;
    if (none(i)) return nullptr;
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != at::kByte || t->device() != dev || !t->is_contiguous() || t->numel() < need) return fail(), nullptr;
    *bytes = t->numel();
    return *bytes ? t->data_ptr() : nullptr;
  }
};

int type_code(at::ScalarType t) { return t == at::kFloat ? TQ_F32 : t == at::kBFloat16 ? TQ_BF16 : t == at::kHalf ? TQ_F16 : -1; }
int32_t dim32(int64_t x) { return x > INT32_MAX ? INT32_MAX : (int32_t)x; }

// The type and device that the first tensor settles.
const at::Tensor* leader(Args& a, int i) {
  const at::Tensor* t = a.tensor(i);
  if (!t || !t->is_cuda() || type_code(t->scalar_type()) < 0) return a.fail();
  a.dev = t->device();
  return t;
}

struct Cache {
  int64_t pages;
  int32_t heads, page, dim;
  at::ScalarType type;
  void *k, *v;
};
bool cache(Args& a, int i, Cache* c) {
  const at::Tensor* t = a.tensor(i);
  if (!t || t->dim() != 4 || (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kHalf)) return a.ok = false;
  const auto s = t->sizes();
  c->type = t->scalar_type();
  c->k = a.full(i, c->type, s);
  c->v = a.full(i + 1, c->type, {s[0], s[1], s[3], s[2]});
  c->pages = s[0], c->heads = dim32(s[1]), c->page = dim32(s[2]), c->dim = dim32(s[3]);
  return a.ok;
}

template <typename ARGS>
PyObject* finish(const Args& a, int (*call)(const ARGS*, void*), const ARGS& args, PyObject* out) {
  PyObject* index = PyLong_FromLong(a.dev.index());
  PyObject* stream = index ? PyObject_CallOneArg(g_stream, index) : nullptr;
  Py_XDECREF(index);
  if (!stream) return nullptr;
  void* s = PyLong_AsVoidPtr(stream);
  Py_DECREF(stream);
  if (PyErr_Occurred()) return nullptr;
  const c10::DeviceGuard guard(a.dev);  // the tensors' device, whatever the current one is
  const int status = call(&args, s);
  if (status != TQ_OK) return PyLong_FromLong(status);
  Py_INCREF(out);
  return out;
}

// q, k, v, positions, slots, inv_freq, k_cache, v_cache, q_norm, k_norm, eps, layout, rope_scale, out, bad_flag
PyObject* rope_append(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  Args a{argv, n};
  const at::Tensor* q = n == 15 ? leader(a, 0) : nullptr;
  if (!q) Py_RETURN_NONE;
  const auto type = q->scalar_type();
  tq_rope_append_args r{};
  at::IntArrayRef qs, ks, vs;
  Cache c;
  r.q = a.heads(0, type, &qs, &r.q_token, &r.q_head);
  if (a.ok) r.k = a.heads(1, type, &ks, &r.k_token, &r.k_head);
  if (a.ok) r.v = a.heads(2, type, &vs, &r.v_token, &r.v_head);
  if (!a.ok || !cache(a, 6, &c)) Py_RETURN_NONE;
  if (ks != vs || ks[0] != qs[0] || ks[1] != c.heads || ks[2] != qs[2] || c.dim != qs[2]) Py_RETURN_NONE;
  int64_t half = 0;
  if (!a.none(5)) {
    const at::Tensor* f = a.tensor(5);
    if (!f) Py_RETURN_NONE;
    half = f->numel();
    r.inv_freq = static_cast<const double*>(a.full(5, at::kDouble, {half}));
  }
  r.positions = static_cast<const int32_t*>(a.some(3, at::kInt, {qs[0]}));
  r.slots = static_cast<const int64_t*>(a.full(4, at::kLong, {qs[0]}));
  r.q_norm = static_cast<const float*>(a.some(8, at::kFloat, {qs[2]}));
  r.k_norm = static_cast<const float*>(a.some(9, at::kFloat, {qs[2]}));
  r.q_out = a.full(13, c.type, qs);
  r.bad_flag = static_cast<int32_t*>(a.some(14, at::kInt, {1}));
  r.eps = a.real(10), r.layout = a.integer32(11), r.rope_scale = a.real(12);
  if (!a.ok || half > INT32_MAX / 2) Py_RETURN_NONE;
  r.k_cache = c.k, r.v_cache = c.v, r.tokens = qs[0], r.pages = c.pages, r.heads = dim32(qs[1]), r.kv_heads = c.heads, r.dim = c.dim;
  r.rot = (int32_t)(2 * half), r.page = c.page, r.in_type = type_code(type), r.cache_type = type_code(c.type);
  return finish(a, tq_rope_append, r, argv[13]);
}

// q, k_cache, v_cache, block_table, kv_len, cu, scale, window, max_len, out, lse, ws, bad_flag
PyObject* paged_attn(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  Args a{argv, n};
  const at::Tensor* q = n == 13 ? leader(a, 0) : nullptr;
  if (!q) Py_RETURN_NONE;
  tq_paged_attn_args r{};
  at::IntArrayRef qs;
  Cache c;
  r.q = a.heads(0, q->scalar_type(), &qs, &r.q_token, &r.q_head);
  if (!a.ok || !cache(a, 1, &c) || c.type != q->scalar_type() || c.dim != qs[2]) Py_RETURN_NONE;
  const at::Tensor *table = a.tensor(3), *out = a.tensor(9);
  if (!table || !out || table->dim() != 2 || table->scalar_type() != at::kInt || table->device() != a.dev) Py_RETURN_NONE;
  r.seqs = table->size(0), r.table_width = table->size(1);
  if (table->stride(1) != 1 && r.table_width > 1) Py_RETURN_NONE;
  r.table_stride = r.seqs > 1 ? table->stride(0) : r.table_width;
  r.block_table = static_cast<const int32_t*>(table->data_ptr());
  r.kv_len = static_cast<const int32_t*>(a.full(4, at::kInt, {r.seqs}));
  r.cu = static_cast<const int32_t*>(a.some(5, at::kInt, {r.seqs + 1}));
  r.out_type = type_code(out->scalar_type());
  r.out = a.full(9, out->scalar_type(), qs);
  r.lse = static_cast<float*>(a.some(10, at::kFloat, {qs[0], qs[1]}));
  r.bad_flag = static_cast<int32_t*>(a.some(12, at::kInt, {1}));
  r.scale = a.real(6, 1 / std::sqrt((double)qs[2])), r.window = a.integer32(7), r.max_len = a.integer(8);
  r.tokens = qs[0], r.pages = c.pages, r.heads = dim32(qs[1]), r.kv_heads = c.heads, r.dim = c.dim, r.page = c.page;
  r.workspace = a.workspace(11, a.none(11) ? 0 : tq_paged_attn_workspace_bytes(r.tokens, r.seqs, r.heads, r.kv_heads, r.dim), &r.workspace_bytes);
  if (!a.ok || r.out_type < 0) Py_RETURN_NONE;
  r.k_cache = c.k, r.v_cache = c.v, r.cache_type = type_code(c.type);
  return finish(a, tq_paged_attn, r, argv[9]);
}

// q, k, v, g, beta, state, cu, slots, scale, l2norm, eps, max_len, out, state_out, ws, bad_flag
PyObject* gdn(PyObject*, PyObject* const* argv, Py_ssize_t n) {
  Args a{argv, n};
  const at::Tensor* q = n == 16 ? leader(a, 0) : nullptr;
  if (!q) Py_RETURN_NONE;
  const auto type = q->scalar_type();
  tq_gdn_args r{};
  at::IntArrayRef qs, ks, vs;
  r.q = a.heads(0, type, &qs, &r.q_token, &r.q_head);
  if (a.ok) r.k = a.heads(1, type, &ks, &r.k_token, &r.k_head);
  if (a.ok) r.v = a.heads(2, type, &vs, &r.v_token, &r.v_head);
  const at::Tensor *state = a.ok ? a.tensor(5) : nullptr, *out = a.ok ? a.tensor(12) : nullptr;
  if (!a.ok || ks != qs || vs[0] != qs[0] || state->dim() != 4) Py_RETURN_NONE;
  r.states = state->size(0);
  const int64_t shape[4] = {r.states, vs[1], qs[2], vs[2]};
  r.state = static_cast<const float*>(a.full(5, at::kFloat, shape));
  r.state_out = static_cast<float*>(a.none(13) ? const_cast<float*>(r.state) : a.full(13, at::kFloat, shape));
  r.seqs = qs[0];
  if (!a.none(6)) {
    const at::Tensor* cu = a.tensor(6);
    if (!cu || cu->dim() != 1 || cu->size(0) < 1) Py_RETURN_NONE;
    r.seqs = cu->size(0) - 1;
    r.cu = static_cast<const int32_t*>(a.full(6, at::kInt, {r.seqs + 1}));
  }
  r.slots = static_cast<const int32_t*>(a.some(7, at::kInt, {r.seqs}));
  r.g = static_cast<const float*>(a.full(3, at::kFloat, {qs[0], vs[1]}));
  r.beta = static_cast<const float*>(a.full(4, at::kFloat, {qs[0], vs[1]}));
  r.out_type = type_code(out->scalar_type());
  r.out = a.full(12, out->scalar_type(), vs);
  r.bad_flag = static_cast<int32_t*>(a.some(15, at::kInt, {1}));
  r.scale = a.real(8, 1 / std::sqrt((double)qs[2])), r.l2norm = a.integer32(9), r.eps = a.real(10), r.max_len = a.integer(11);
  r.tokens = qs[0], r.k_heads = dim32(qs[1]), r.v_heads = dim32(vs[1]), r.dk = dim32(qs[2]), r.dv = dim32(vs[2]);
  r.workspace = a.workspace(14, a.none(14) ? 0 : tq_gdn_workspace_bytes(r.tokens, r.seqs, r.max_len, r.v_heads, r.dk, r.dv), &r.workspace_bytes);
  if (!a.ok || r.out_type < 0) Py_RETURN_NONE;
  r.in_type = type_code(type);
  return finish(a, tq_gdn, r, argv[12]);
}

// A C++ exception must not pass through the interpreter.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* argv, Py_ssize_t n) {
  try {
    return F(self, argv, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "tq: unknown error");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<F>));
}

PyMethodDef g_methods[] = {{"rope_append", method<rope_append>(), METH_FASTCALL, nullptr},
                           {"paged_attn", method<paged_attn>(), METH_FASTCALL, nullptr},
                           {"gdn", method<gdn>(), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* c = PyImport_ImportModule("torch._C");
  if (!c) return nullptr;
  g_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_DECREF(c);
  PyObject* m = g_stream ? PyModule_Create(&g_module) : nullptr;
  if (m && PyModule_AddStringConstant(m, "torch_version", TQ_TORCH_VERSION) != 0) Py_CLEAR(m);  // whose headers this was built with
  return m;
}
