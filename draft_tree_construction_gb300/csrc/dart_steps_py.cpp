// dart_steps_py.cpp -- the usual calls of the steps around a tree and behind a
// verified one, without the interpreter: tensors in, the C entry point, tensors out.
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
decltype(&dart_logits_sample) logits_sample = nullptr;            // these by bind_verified()
decltype(&dart_tree_accept) tree_accept = nullptr;
decltype(&dart_kv_keep) kv_keep = nullptr;
decltype(&dart_attention_weights) attention_weights = nullptr;
decltype(&dart_kv_evict) kv_evict = nullptr;
decltype(&dart_kv_keep_scored) kv_keep_scored = nullptr;
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

// -------------------------------------------------- behind a verified tree

// An error word: absent, or at least one packed integer.
bool error_word(const Tensor* t) { return !t || (packed(*t) && t->numel() >= 1 && t->is_contiguous()); }
bool ints(const Tensor* t, int64_t B, int64_t n) {             // contiguous int32 [B, n]
  return t && t->scalar_type() == at::kInt && t->dim() == 2 && t->size(0) == B && t->size(1) == n && t->is_contiguous();
}

// (logits, uniforms, temperature, top_k, top_p, min_p) -> (tokens, probs)
PyObject* sample(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 6) Py_RETURN_NONE;
  Taker take;
  const Tensor *z = take(args[0]), *u = take(args[1]), *temperature = take(args[2]), *top_k = take(args[3]),
               *top_p = take(args[4]), *min_p = take(args[5]);
  if (!take.ok || !logits_sample || !z || !u || z->dim() != 3 || z->numel() == 0) Py_RETURN_NONE;
  const int64_t B = z->size(0), R = z->size(1), V = z->size(2), stride = row_stride(*z);
  const int code = dtype_code(z->scalar_type());
  if (code < 0 || stride < 0 || B > INT_MAX || R > INT_MAX || V > INT_MAX || u->scalar_type() != at::kFloat ||
      u->dim() != 2 || u->size(0) != B || u->size(1) != R || !u->is_contiguous() || !is(temperature, at::kFloat, B) ||
      !is(top_k, at::kInt, B) || !is(top_p, at::kFloat, B) || !is(min_p, at::kFloat, B))
    Py_RETURN_NONE;
  Tensor tokens = at::empty({B, R}, u->options().dtype(at::kInt)), probs = at::empty({B, R}, u->options());
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = logits_sample(z->data_ptr(), int(B), int(R), int(V), stride, code, at_of<float>(u), at_of<float>(temperature),
                     at_of<int32_t>(top_k), at_of<float>(top_p), at_of<float>(min_p), at_of<int32_t>(&tokens),
                     at_of<float>(&probs), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_logits_sample");
  return Py_BuildValue("NN", THPVariable_Wrap(tokens), THPVariable_Wrap(probs));
  END_HANDLE_TH_ERRORS
}

// (picks, tokens, parents, depth) -> (path, counts, tokens)
PyObject* accept(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 4) Py_RETURN_NONE;
  Taker take;
  const Tensor *picks = take(args[0]), *tokens = take(args[1]), *parents = take(args[2]);
  if (!take.ok || !tree_accept || !picks || !tokens || !parents || tokens->dim() != 2 || tokens->numel() == 0 ||
      !PyLong_Check(args[3]))
    Py_RETURN_NONE;
  const int64_t B = tokens->size(0), N = tokens->size(1);
  const long depth = PyLong_AsLong(args[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (!ints(tokens, B, N) || !ints(parents, B, N) || !ints(picks, B, N + 1) || B > INT_MAX || N > INT_MAX ||
      depth < 0 || depth > N)
    Py_RETURN_NONE;
  Tensor path = at::empty({B, depth + 1}, tokens->options()), counts = at::empty({B}, tokens->options()),
         out = at::empty({B, depth + 1}, tokens->options());
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = tree_accept(at_of<int32_t>(picks), at_of<int32_t>(tokens), at_of<int32_t>(parents), int(B), int(N), int(depth),
                   at_of<int32_t>(&path), at_of<int32_t>(&counts), at_of<int32_t>(&out), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_tree_accept");
  return Py_BuildValue("NNN", THPVariable_Wrap(path), THPVariable_Wrap(counts), THPVariable_Wrap(out));
  END_HANDLE_TH_ERRORS
}

// B of lengths [B], or -1.
int64_t lengths_of(const Tensor* lengths) {
  if (!lengths || lengths->dim() != 1) return -1;
  const int64_t B = lengths->size(0);
  return B > 0 && B < INT_MAX && is(lengths, at::kInt, B) && lengths->is_contiguous() ? B : -1;
}

// The (sequence, head) strides of scores [B, heads, width]: false where the binding has to look.
bool scores_of(const Tensor* t, int64_t B, int64_t heads, int64_t* seq, int64_t* head) {
  if (!t || t->dim() != 3 || t->size(0) != B || t->size(1) != heads || t->scalar_type() != at::kFloat ||
      t->numel() == 0 || t->size(2) > INT_MAX || (t->size(2) > 1 && t->stride(2) != 1))
    return false;
  const int64_t width = t->size(2);
  *head = heads > 1 ? t->stride(1) : width;
  *seq = B > 1 ? t->stride(0) : heads * *head;
  return *head >= width && (B <= 1 || *seq >= *head * (heads - 1) + width);
}

// (k_cache, v_cache, pages, lengths, path, counts, scores, starts, device_err) -> lengths
PyObject* keep(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 9) Py_RETURN_NONE;
  Taker take;
  const Tensor *k_cache = take(args[0]), *v_cache = take(args[1]), *pages = take(args[2]), *lengths = take(args[3]),
               *path = take(args[4]), *counts = take(args[5]), *scores = take(args[6]), *starts = take(args[7]),
               *err = take(args[8]);
  const int64_t B = lengths_of(lengths);
  dart_cache_t c;
  int64_t s_seq = 0, s_head = 0;
  if (!take.ok || !kv_keep || !kv_keep_scored || B < 0 || !path || !counts ||
      !cache_of(k_cache, v_cache, pages, B, &c) || !error_word(err) || !is(counts, at::kInt, B) || path->dim() != 2 ||
      path->size(0) != B || path->size(1) < 1 || path->size(1) > INT_MAX || path->scalar_type() != at::kInt ||
      (path->size(1) > 1 && path->stride(1) != 1) || (scores == nullptr) != (starts == nullptr) ||
      (scores && (!scores_of(scores, B, c.heads, &s_seq, &s_head) || !is(starts, at::kInt, B + 1))))
    Py_RETURN_NONE;
  const int64_t width = path->size(1), step = B > 1 ? path->stride(0) : width;
  if (step < width) Py_RETURN_NONE;
  Tensor out = at::empty({B}, lengths->options());
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  if (scores)
    rc = kv_keep_scored(&c, at_of<int32_t>(lengths), at_of<int32_t>(path), step, at_of<int32_t>(counts), int(B),
                        int(width), at_of<int32_t>(starts), at_of<float>(scores), s_seq, s_head, int(scores->size(2)),
                        at_of<int32_t>(&out), at_of<uint32_t>(err), stream);
  else
    rc = kv_keep(&c, at_of<int32_t>(lengths), at_of<int32_t>(path), step, at_of<int32_t>(counts), int(B), int(width),
                 at_of<int32_t>(&out), at_of<uint32_t>(err), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, scores ? "dart_kv_keep_scored" : "dart_kv_keep");
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// (q, k_cache, pages, lengths, starts, lse, scores, mask, scale, device_err) -> scores
PyObject* weights(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 10) Py_RETURN_NONE;
  Taker take;
  const Tensor *q = take(args[0]), *k_cache = take(args[1]), *pages = take(args[2]), *lengths = take(args[3]),
               *starts = take(args[4]), *lse = take(args[5]), *scores = take(args[6]), *mask = take(args[7]),
               *err = take(args[9]);
  if (!take.ok || !attention_weights || !q || !lse || q->dim() != 3 || q->numel() == 0) Py_RETURN_NONE;
  const int64_t B = sequences(lengths, starts), T = q->size(0), q_heads = q->size(1);
  dart_cache_t c;
  Heads hq;
  int64_t s_seq, s_head;
  if (B < 0 || T > INT_MAX || q_heads > INT_MAX || !cache_of(k_cache, k_cache, pages, B, &c) ||
      !hq.fit(*q, T, q_heads, c.dim, k_cache->scalar_type(), true) || q_heads % c.heads != 0 ||
      lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != T || lse->size(1) != q_heads ||
      !lse->is_contiguous() || !scores_of(scores, B, c.heads, &s_seq, &s_head) || !error_word(err))
    Py_RETURN_NONE;
  int64_t N = 0;
  if (mask) {
    if (!packed(*mask) || mask->dim() != 3 || mask->size(0) != B || mask->size(2) != (mask->size(1) + 31) / 32 ||
        !mask->is_contiguous() || mask->size(1) > INT_MAX)
      Py_RETURN_NONE;
    N = mask->size(1);
  }
  double scale = std::pow(double(c.dim), -0.5);
  if (args[8] != Py_None) {
    scale = PyFloat_AsDouble(args[8]);
    if (PyErr_Occurred()) return nullptr;
  }
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = attention_weights(q->data_ptr(), hq.token, hq.head, int(q_heads), int(T), int(B), at_of<int32_t>(lengths),
                         at_of<int32_t>(starts), at_of<uint32_t>(mask), int(N), float(scale), &c, at_of<float>(lse),
                         at_of<float>(scores), s_seq, s_head, int(scores->size(2)), at_of<uint32_t>(err), stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_attention_weights");
  return Py_NewRef(args[6]);
  END_HANDLE_TH_ERRORS
}

// (k_cache, v_cache, pages, lengths, scores, keep, first, last, device_err) -> (lengths, index)
PyObject* evict(PyObject*, PyObject* const* args, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 9) Py_RETURN_NONE;
  Taker take;
  const Tensor *k_cache = take(args[0]), *v_cache = take(args[1]), *pages = take(args[2]), *lengths = take(args[3]),
               *scores = take(args[4]), *err = take(args[8]);
  const int64_t B = lengths_of(lengths);
  dart_cache_t c;
  int64_t s_seq, s_head, n[3];
  if (!take.ok || !kv_evict || B < 0 || !cache_of(k_cache, v_cache, pages, B, &c) ||
      !scores_of(scores, B, c.heads, &s_seq, &s_head) || !error_word(err))
    Py_RETURN_NONE;
  for (int i = 0; i < 3; ++i) {
    if (!PyLong_Check(args[5 + i])) Py_RETURN_NONE;
    n[i] = PyLong_AsLongLong(args[5 + i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
  }
  if (n[0] < 1 || n[0] > INT_MAX || n[1] < 0 || n[2] < 0 || n[1] > n[0] || n[2] > n[0] - n[1]) Py_RETURN_NONE;
  Tensor out = at::empty({B}, lengths->options()), index = at::empty({B, c.heads, n[0]}, lengths->options());
  int rc;
  void* const stream = current_stream(take.device);
  Py_BEGIN_ALLOW_THREADS
  rc = kv_evict(&c, at_of<int32_t>(lengths), int(B), at_of<float>(scores), s_seq, s_head, int(scores->size(2)),
                int(n[0]), int(n[1]), int(n[2]), at_of<int32_t>(&index), at_of<int32_t>(&out), at_of<uint32_t>(err),
                stream);
  Py_END_ALLOW_THREADS
  if (rc != DART_OK) return failed(rc, "dart_kv_evict");
  return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(index));
  END_HANDLE_TH_ERRORS
}

// (the addresses of dart_logits_sample, dart_tree_accept, dart_kv_keep, dart_attention_weights, dart_kv_evict and
// dart_kv_keep_scored)
PyObject* bind_verified(PyObject*, PyObject* const* args, Py_ssize_t count) {
  void* at[6];
  if (count != 6) {
    PyErr_SetString(PyExc_TypeError, "bind_verified takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  logits_sample = reinterpret_cast<decltype(logits_sample)>(at[0]);
  tree_accept = reinterpret_cast<decltype(tree_accept)>(at[1]);
  kv_keep = reinterpret_cast<decltype(kv_keep)>(at[2]);
  attention_weights = reinterpret_cast<decltype(attention_weights)>(at[3]);
  kv_evict = reinterpret_cast<decltype(kv_evict)>(at[4]);
  kv_keep_scored = reinterpret_cast<decltype(kv_keep_scored)>(at[5]);
  Py_RETURN_NONE;
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
                         {"sample", method(sample), METH_FASTCALL, nullptr},
                         {"accept", method(accept), METH_FASTCALL, nullptr},
                         {"keep", method(keep), METH_FASTCALL, nullptr},
                         {"weights", method(weights), METH_FASTCALL, nullptr},
                         {"evict", method(evict), METH_FASTCALL, nullptr},
                         {"bind", method(bind), METH_FASTCALL, nullptr},
                         {"bind_verified", method(bind_verified), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_steps_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__steps_native() { return PyModule_Create(&module); }
