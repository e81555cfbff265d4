// dart_steps_py.cpp -- the usual calls of the steps around a tree, without the
// interpreter: tensors in, the C entry point, tensors out.
//
// Checks and arguments in Python cost 9 to 13 us a call on a Grace core (an
// adjustment with everything 20), longer than many of these kernels run; here
// they cost one or two.  A function takes its arguments only when everything is
// as the Python binding would accept it, on the current device and stream;
// otherwise it returns None, nothing has happened, and the caller goes the
// binding's way, which handles the rest and finds the words for what is wrong.
// Once the entry point has been called, its answer is the call's: an error is
// raised here, because part of the work may have been launched.
#include <Python.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "darttree.h"

namespace {

using at::Tensor;

// The library's entry points, handed over by bind().
decltype(&dart_logits_adjust) logits_adjust = nullptr;
decltype(&dart_kv_append) kv_append = nullptr;
decltype(&dart_tree_attention) tree_attention = nullptr;
decltype(&dart_attention_workspace_bytes) workspace_bytes = nullptr;
PyObject* check = nullptr;          // check(code, name) raises the package's error; also from bind()

PyObject* failed(int rc, const char* name) {
  PyObject* const r = PyObject_CallFunction(check, "is", rc, name);
  if (r) PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", name, rc);
  Py_XDECREF(r);
  return nullptr;
}

// Takes tensors that lie on the current device; ok turns false at the first argument that does not.
struct Taker {
  int device = c10::cuda::current_device();
  bool ok = true;
  const Tensor* operator()(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (THPVariable_Check(o)) {
      const Tensor& t = THPVariable_Unpack(o);
      if (t.defined() && t.is_cuda() && t.get_device() == device) return &t;
    }
    ok = false;
    return nullptr;
  }
};

bool is(const Tensor* t, at::ScalarType type, int64_t n) {      // absent, or a vector of n
  return !t || (t->scalar_type() == type && t->dim() == 1 && t->size(0) == n && (n <= 1 || t->stride(0) == 1));
}
bool packed(const Tensor& t) { return t.scalar_type() == at::kInt || t.scalar_type() == at::kUInt32; }
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <typename T> T* at_of(const Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }
int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? DART_F32 : t == at::kHalf ? DART_F16 : t == at::kBFloat16 ? DART_BF16 : -1;
}
void* current_stream(int device) { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream(); }

// Elements between the starts of evenly spaced rows of a [B, R, V] tensor, -1 if they are not.
int64_t row_stride(const Tensor& t) {
  const int64_t B = t.size(0), R = t.size(1), V = t.size(2);
  if (V > 1 && t.stride(2) != 1) return -1;
  if (B * R <= 1) return V;
  const int64_t step = R > 1 ? t.stride(1) : t.stride(0);
  if (R > 1 && B > 1 && t.stride(0) != step * R) return -1;
  return step >= V ? step : -1;
}

// (logits, history, lengths, repetition, presence, frequency, bias ids, bias values, allowed, tokens, mask, out)
PyObject* adjust(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 12) Py_RETURN_NONE;
  Taker take;
  const Tensor* z = take(args[0]);
  const Tensor *history = take(args[1]), *lengths = take(args[2]), *repetition = take(args[3]),
               *presence = take(args[4]), *frequency = take(args[5]), *ids = take(args[6]), *vals = take(args[7]),
               *allowed = take(args[8]), *tokens = take(args[9]), *mask = take(args[10]), *out = take(args[11]);
  if (!take.ok || !z || z->dim() != 3 || z->numel() == 0) Py_RETURN_NONE;
  const int64_t B = z->size(0), R = z->size(1), V = z->size(2), stride = row_stride(*z);
  const int code = dtype_code(z->scalar_type());
  if (code < 0 || stride < 0 || B > INT_MAX || R > INT_MAX || V > INT_MAX) Py_RETURN_NONE;
  dart_adjust_t a = {};
  if (history) {
    if (history->dim() != 2 || history->size(0) != B || history->scalar_type() != at::kInt) Py_RETURN_NONE;
    const int64_t width = history->size(1), step = B > 1 ? history->stride(0) : width;
    if ((width > 1 && history->stride(1) != 1) || step < width || width > INT_MAX) Py_RETURN_NONE;
    a.history = at_of<int32_t>(history);
    a.history_width = int32_t(width);
    a.history_stride = step;
  } else if (lengths) {
    Py_RETURN_NONE;
  }
  if (!is(lengths, at::kInt, B) || !is(repetition, at::kFloat, B) || !is(presence, at::kFloat, B) ||
      !is(frequency, at::kFloat, B))
    Py_RETURN_NONE;
  a.history_len = at_of<int32_t>(lengths);
  a.repetition = at_of<float>(repetition);
  a.presence = at_of<float>(presence);
  a.frequency = at_of<float>(frequency);
  if (ids || vals) {
    if (!ids || !vals || ids->dim() != 2 || ids->size(0) != B || ids->scalar_type() != at::kInt ||
        vals->scalar_type() != at::kFloat || vals->sizes() != ids->sizes() || !ids->is_contiguous() ||
        !vals->is_contiguous() || ids->size(1) > INT_MAX)
      Py_RETURN_NONE;
    a.bias_ids = at_of<int32_t>(ids);
    a.bias_vals = at_of<float>(vals);
    a.bias_count = int32_t(ids->size(1));
  }
  if (allowed) {
    const int64_t words = (V + 31) / 32;
    const bool rows = allowed->dim() == 3;
    if (!packed(*allowed) || (!rows && allowed->dim() != 2) || allowed->size(0) != B || allowed->size(-1) != words ||
        (rows && allowed->size(1) != R) || (words > 1 && allowed->stride(-1) != 1))
      Py_RETURN_NONE;
    a.allowed = at_of<uint32_t>(allowed);
    a.allowed_seq_stride = B > 1 ? allowed->stride(0) : 0;
    a.allowed_row_stride = rows && R > 1 ? allowed->stride(1) : 0;
  }
  if (tokens || mask) {
    if (!tokens || !mask || tokens->dim() != 2 || tokens->size(0) != B || tokens->scalar_type() != at::kInt ||
        !tokens->is_contiguous() || !packed(*mask) || !mask->is_contiguous() || mask->dim() != 3)
      Py_RETURN_NONE;
    const int64_t N = tokens->size(1);
    if (mask->size(0) != B || mask->size(1) != N || mask->size(2) != (N + 31) / 32 || (R != N && R != N + 1))
      Py_RETURN_NONE;
    a.tokens = at_of<int32_t>(tokens);
    a.mask = at_of<uint32_t>(mask);
    a.N = int32_t(N);
  }
  Tensor made;
  int64_t out_stride;
  if (out) {
    if (out->scalar_type() != z->scalar_type() || out->sizes() != z->sizes()) Py_RETURN_NONE;
    out_stride = row_stride(*out);
    if (out_stride < 0 || (out->data_ptr() == z->data_ptr() && out_stride != stride && B * R > 1)) Py_RETURN_NONE;
  } else {
    // rows that keep the input's alignment take whole vectors from end to end
    out_stride = V + (stride - V) % (16 / z->element_size());
    made = at::empty({B, R, out_stride}, z->options());
    if (out_stride != V) made = made.narrow(2, 0, V);
    out = &made;
  }
  int rc;
  void* const stream = current_stream(take.device);
  const void* const from = z->data_ptr();
  void* const to = out->data_ptr();
  Py_BEGIN_ALLOW_THREADS
  rc = logits_adjust(from, int(B), int(R), int(V), stride, code, &a, to, out_stride, stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_logits_adjust");
  return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[11]);
  END_HANDLE_TH_ERRORS
}

// lengths [B] and starts [B + 1]; B, or -1.
int64_t sequences(const Tensor* lengths, const Tensor* starts) {
  if (!lengths || !starts || lengths->dim() != 1) return -1;
  const int64_t B = lengths->size(0);
  return B > 0 && B < INT_MAX && is(lengths, at::kInt, B) && is(starts, at::kInt, B + 1) ? B : -1;
}

// Caches [pages, page, heads, dim] with their page table [B, width].
bool cache_of(const Tensor* k, const Tensor* v, const Tensor* table, int64_t B, dart_cache_t* c) {
  if (!k || !v || !table || k->dim() != 4 || v->sizes() != k->sizes() || v->scalar_type() != k->scalar_type() ||
      table->dim() != 2 || table->size(0) != B || table->scalar_type() != at::kInt || k->numel() == 0 ||
      table->numel() == 0)
    return false;
  const int code = dtype_code(k->scalar_type());
  const int64_t count = k->size(0), page = k->size(1), heads = k->size(2), dim = k->size(3), width = table->size(1);
  const int64_t step = B > 1 ? table->stride(0) : width;
  if ((code != DART_F16 && code != DART_BF16) || (width > 1 && table->stride(1) != 1) || step < width ||
      count > INT_MAX || page > INT_MAX || heads > INT_MAX || width > INT_MAX || page < 8 || page & 7 || dim < 8 ||
      dim > 128 || dim & 7 || k->stride(3) != 1 || v->stride(3) != 1)
    return false;
  int64_t st[6] = {k->stride(0), k->stride(1), k->stride(2), v->stride(0), v->stride(1), v->stride(2)};
  if (count <= 1) st[0] = st[3] = 8;          // a dimension of one is never stepped along
  if (heads == 1) st[2] = st[5] = 8;
  for (int64_t s : st)
    if (s == 0 || s & 7) return false;        // 0: an expanded tensor cannot be written
  if (!aligned(k->data_ptr()) || !aligned(v->data_ptr())) return false;
  *c = dart_cache_t{k->data_ptr(), v->data_ptr(), st[0], st[1], st[2], st[3], st[4], st[5], at_of<int32_t>(table),
                    step, int32_t(width), int32_t(count), int32_t(page), int32_t(heads), int32_t(dim), code};
  return true;
}

// A [T, heads, dim] tensor of vectors and its strides; one that is written must not share memory between elements.
struct Heads {
  int64_t token = 0, head = 0;
  bool fit(const Tensor& t, int64_t T, int64_t heads, int64_t dim, at::ScalarType type, bool written = false) {
    if (t.dim() != 3 || t.size(0) != T || t.size(1) != heads || t.size(2) != dim || t.scalar_type() != type ||
        t.stride(2) != 1)
      return false;
    token = T > 1 ? t.stride(0) : 0;
    head = heads > 1 ? t.stride(1) : 0;
    if (written && ((T > 1 && token == 0) || (heads > 1 && head == 0))) return false;
    return ((token | head) & 7) == 0 && aligned(t.data_ptr());
  }
};

// (q, k, v, k_cache, v_cache, pages, lengths, starts, turns, address of the dart_rotary_t, offsets, q_weight,
// k_weight, eps, out, device_err); turns is None without a rotary
PyObject* append(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 16) Py_RETURN_NONE;
  Taker take;
  const Tensor *q = take(args[0]), *k = take(args[1]), *v = take(args[2]), *k_cache = take(args[3]),
               *v_cache = take(args[4]), *pages = take(args[5]), *lengths = take(args[6]), *starts = take(args[7]),
               *turns = take(args[8]), *offsets = take(args[10]), *q_weight = take(args[11]),
               *k_weight = take(args[12]), *out = take(args[14]), *err = take(args[15]);
  if (!take.ok || !q || !k || !v || k->dim() != 3 || q->dim() != 3 || q->numel() == 0 || k->numel() == 0)
    Py_RETURN_NONE;
  const int64_t B = sequences(lengths, starts), T = k->size(0), q_heads = q->size(1);
  dart_cache_t c;
  if (B < 0 || T > INT_MAX || q_heads > INT_MAX || !cache_of(k_cache, v_cache, pages, B, &c)) Py_RETURN_NONE;
  const at::ScalarType type = k_cache->scalar_type();
  const int64_t dim = c.dim;
  Heads hq, hk, hv, ho;
  if (!hq.fit(*q, T, q_heads, dim, type) || !hk.fit(*k, T, c.heads, dim, type) || !hv.fit(*v, T, c.heads, dim, type))
    Py_RETURN_NONE;
  if (out) {
    if (!ho.fit(*out, T, q_heads, dim, type, true) ||
        (out->data_ptr() == q->data_ptr() && (ho.token != hq.token || ho.head != hq.head)))
      Py_RETURN_NONE;
  }
  if (!is(offsets, at::kInt, T) || !is(q_weight, type, dim) || !is(k_weight, type, dim)) Py_RETURN_NONE;
  if (err && (!packed(*err) || err->numel() < 1 || !err->is_contiguous())) Py_RETURN_NONE;
  const dart_rotary_t* rotary = nullptr;
  if (turns) {
    rotary = static_cast<const dart_rotary_t*>(PyLong_AsVoidPtr(args[9]));
    if (PyErr_Occurred()) return nullptr;
    if (!rotary || rotary->rot > dim) Py_RETURN_NONE;
  }
  const double eps = PyFloat_AsDouble(args[13]);
  if (PyErr_Occurred()) return nullptr;
  Tensor made;
  if (!out) {
    made = at::empty({T, q_heads, dim}, q->options());
    out = &made;
    ho.token = q_heads * dim;
    ho.head = dim;
  }
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = kv_append(q->data_ptr(), hq.token, hq.head, int(q_heads), k->data_ptr(), hk.token, hk.head, v->data_ptr(),
                 hv.token, hv.head, int(T), int(B), at_of<int32_t>(lengths), at_of<int32_t>(starts),
                 at_of<int32_t>(offsets), rotary, at_of<void>(q_weight), at_of<void>(k_weight), float(eps), &c,
                 out->data_ptr(), ho.token, ho.head, at_of<uint32_t>(err), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_kv_append");
  return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[14]);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, v_cache, pages, lengths, starts, mask, scale, out, lse, workspace) -> (out, lse, workspace)
PyObject* attend(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 11) Py_RETURN_NONE;
  Taker take;
  const Tensor *q = take(args[0]), *k_cache = take(args[1]), *v_cache = take(args[2]), *pages = take(args[3]),
               *lengths = take(args[4]), *starts = take(args[5]), *mask = take(args[6]), *out = take(args[8]),
               *workspace = take(args[10]);
  if (!take.ok || !q || q->dim() != 3 || q->numel() == 0) Py_RETURN_NONE;
  const int64_t B = sequences(lengths, starts), T = q->size(0), q_heads = q->size(1);
  dart_cache_t c;
  if (B < 0 || T > INT_MAX || q_heads > INT_MAX || !cache_of(k_cache, v_cache, pages, B, &c)) Py_RETURN_NONE;
  const at::ScalarType type = k_cache->scalar_type();
  const int64_t dim = c.dim;
  Heads hq, ho;
  if (!hq.fit(*q, T, q_heads, dim, type) || q_heads % c.heads != 0) Py_RETURN_NONE;
  int64_t N = 0;
  if (mask) {
    if (!packed(*mask) || mask->dim() != 3 || mask->size(0) != B || mask->size(2) != (mask->size(1) + 31) / 32 ||
        !mask->is_contiguous() || mask->size(1) > INT_MAX)
      Py_RETURN_NONE;
    N = mask->size(1);
  }
  double scale = 0.0;
  if (args[7] == Py_None) {
    scale = std::pow(double(dim), -0.5);
  } else {
    scale = PyFloat_AsDouble(args[7]);
    if (PyErr_Occurred()) return nullptr;
  }
  if (out && (!ho.fit(*out, T, q_heads, dim, type, true) || out->data_ptr() == q->data_ptr())) Py_RETURN_NONE;
  const int wants_lse = PyObject_IsTrue(args[9]);
  if (wants_lse < 0) return nullptr;
  const size_t need = workspace_bytes(int(T), int(B), int(q_heads), c.heads, c.dim);
  if (need == 0) Py_RETURN_NONE;
  if (workspace && (!workspace->is_contiguous() || workspace->nbytes() < need)) Py_RETURN_NONE;
  Tensor made, made_lse, made_workspace;
  if (!out) {
    made = at::empty({T, q_heads, dim}, q->options());
    out = &made;
    ho.token = q_heads * dim;
    ho.head = dim;
  }
  if (!workspace) {
    made_workspace = at::empty({int64_t(need)}, q->options().dtype(at::kByte));
    made_workspace.narrow(0, 0, 256).zero_();
    workspace = &made_workspace;
  }
  if (wants_lse) made_lse = at::empty({T, q_heads}, q->options().dtype(at::kFloat));
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = tree_attention(q->data_ptr(), hq.token, hq.head, int(q_heads), int(T), int(B), at_of<int32_t>(lengths),
                      at_of<int32_t>(starts), at_of<uint32_t>(mask), int(N), float(scale), &c, out->data_ptr(),
                      ho.token, ho.head, wants_lse ? static_cast<float*>(made_lse.data_ptr()) : nullptr,
                      workspace->data_ptr(), workspace->nbytes(), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_tree_attention");
  PyObject* result = PyTuple_New(3);
  if (!result) return nullptr;
  PyTuple_SET_ITEM(result, 0, made.defined() ? THPVariable_Wrap(made) : Py_NewRef(args[8]));
  PyTuple_SET_ITEM(result, 1, wants_lse ? THPVariable_Wrap(made_lse) : Py_NewRef(Py_None));
  PyTuple_SET_ITEM(result, 2, made_workspace.defined() ? THPVariable_Wrap(made_workspace) : Py_NewRef(args[10]));
  return result;
  END_HANDLE_TH_ERRORS
}

// (the addresses of dart_logits_adjust, dart_kv_append, dart_tree_attention and
// dart_attention_workspace_bytes, then what raises the package's error)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* at[4];
  if (count != 5 || !PyCallable_Check(args[4])) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses and a function");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  logits_adjust = reinterpret_cast<decltype(logits_adjust)>(at[0]);
  kv_append = reinterpret_cast<decltype(kv_append)>(at[1]);
  tree_attention = reinterpret_cast<decltype(tree_attention)>(at[2]);
  workspace_bytes = reinterpret_cast<decltype(workspace_bytes)>(at[3]);
  PyObject* const old = check;
  check = Py_NewRef(args[4]);
  Py_XDECREF(old);
  Py_RETURN_NONE;
}

template <typename F> PyCFunction method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }
PyMethodDef methods[] = {{"adjust", method(adjust), METH_FASTCALL, nullptr},
                         {"append", method(append), METH_FASTCALL, nullptr},
                         {"attend", method(attend), METH_FASTCALL, nullptr},
                         {"bind", method(bind), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_steps_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__steps_native() { return PyModule_Create(&module); }
