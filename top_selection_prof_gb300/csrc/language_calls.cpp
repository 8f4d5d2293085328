// The calls of language.py: checks of the tensors, outputs from torch's
// allocator on the current stream, and the library's C entries (include/topk.h).
//
// A decoding step's calls take a few microseconds on the GPU; their checks and
// allocations alone took 10 to 16 us in Python (replace_ for one conversation
// 20 us in all), so they are made here.  Each function returns its tensors, or
// the library's status where that is not TOPK_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <cstdarg>
#include <cstdio>
#include <string>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/topk.h"

namespace {

// What a call refuses: a Python exception and its text.
struct Refusal {
  PyObject* type;
  std::string text;
};
[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
  char text[512];
  va_list args;
  va_start(args, format);
  std::vsnprintf(text, sizeof text, format, args);
  va_end(args);
  throw Refusal{type, text};
}

std::string text_of(at::IntArrayRef sizes) {
  std::string s = "(";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + (sizes.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
// dtype code of the tensor that the call's others are checked against.
int code_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return TOPK_F32;
  if (t.scalar_type() == at::kBFloat16) return TOPK_BF16;
  refuse(PyExc_TypeError, "operators take float32 or bfloat16 tensors, got %s", c10::toString(t.scalar_type()));
}
int first(const at::Tensor& t) {
  if (!t.is_cuda()) refuse(PyExc_TypeError, "input must be a CUDA tensor (the engine has no CPU path)");
  return code_of(t);
}
const at::Tensor& like(PyObject* o, at::ScalarType dtype, const at::Device& device, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype || t.device() != device)
    refuse(PyExc_TypeError, "%s must be a %s tensor on %s", name, c10::toString(dtype), device.str().c_str());
  return t;
}
// Distance between the rows of t, which must be (rows, cols) with contiguous rows that do not overlap.
int64_t matrix(const at::Tensor& t, int64_t rows, int64_t cols, const char* name) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(PyExc_ValueError, "%s must have shape (%lld, %lld), got %s", name, static_cast<long long>(rows), static_cast<long long>(cols),
           text_of(t.sizes()).c_str());
  if (t.stride(1) != 1 && cols > 1) refuse(PyExc_ValueError, "%s must be contiguous along its last dimension", name);
  if (rows <= 1) return cols;
  if (t.stride(0) < cols) refuse(PyExc_ValueError, "the rows of %s must not overlap", name);
  return t.stride(0);
}
void two_dims(const at::Tensor& t, const char* name, const char* dims) {
  if (t.dim() != 2) refuse(PyExc_ValueError, "%s must be 2-D %s", name, dims);
}
template <typename T>
const T* vector(PyObject* o, at::ScalarType dtype, const at::Device& device, int64_t n, const char* name) {
  const at::Tensor& t = like(o, dtype, device, name);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be contiguous with %lld values", name, static_cast<long long>(n));
  return static_cast<const T*>(t.data_ptr());
}
// (tokens, k) of contiguous int64; tokens < 0: any.
const at::Tensor& choices(PyObject* o, int64_t tokens, const at::Device& device, const char* name) {
  const at::Tensor& t = like(o, at::kLong, device, name);
  if (t.dim() != 2 || (tokens >= 0 && t.size(0) != tokens) || t.size(1) < 1 || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be contiguous with shape (tokens, k), k >= 1, got %s", name, text_of(t.sizes()).c_str());
  return t;
}
const void* of_places(PyObject* o, const at::Tensor& place, at::ScalarType dtype, const at::Device& device, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = like(o, dtype, device, name);
  if (t.sizes() != place.sizes() || !t.is_contiguous())
    refuse(PyExc_ValueError, "%s must be contiguous with shape %s", name, text_of(place.sizes()).c_str());
  return t.data_ptr();
}
// Rows of contiguous values, (batch, heads, rows, values) or (batch, heads, values).
topk_view_t view(const at::Tensor& t, at::IntArrayRef shape, const char* name) {
  if (t.sizes() != shape) refuse(PyExc_ValueError, "%s must have shape %s, got %s", name, text_of(shape).c_str(), text_of(t.sizes()).c_str());
  if (t.stride(-1) != 1 && shape.back() > 1) refuse(PyExc_ValueError, "%s must be contiguous along its last dimension", name);
  return topk_view_t{t.data_ptr(), t.stride(0), t.stride(1), shape.size() == 4 ? t.stride(2) : 0};
}

int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a whole number", name);
  }
  return v;
}
// A parameter that is a number, or a tensor with one value a row.
template <typename T>
const T* by_row(PyObject* o, at::ScalarType dtype, const at::Device& device, int64_t rows, const char* name, double* number) {
  *number = 0.0;
  if (THPVariable_Check(o)) return vector<T>(o, dtype, device, rows, name);
  *number = PyFloat_AsDouble(o);
  if (*number == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a number or a tensor with one value a row", name);
  }
  return nullptr;
}

// While it lives, other threads run Python, and the device is the tensors'.
class Launch {
 public:
  explicit Launch(const at::Device& device) : guard_(device), state_(PyEval_SaveThread()) {}
  ~Launch() { done(); }
  void done() {
    if (state_) PyEval_RestoreThread(state_);
    state_ = nullptr;
  }

 private:
  c10::cuda::CUDAGuard guard_;
  PyThreadState* state_;
};
// (torch's own allocation without the dispatcher, which takes as long again)
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType dtype, const at::Device& device) {
  return at::Tensor(at::detail::empty_cuda(sizes, dtype, device, std::nullopt));
}
void* stream_of(const at::Device& device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

PyObject* give(int status, std::initializer_list<at::Tensor> out) {
  if (status != TOPK_OK) return PyLong_FromLong(status);
  if (out.size() == 1) return THPVariable_Wrap(*out.begin());
  PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(out.size()));
  if (!tuple) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : out) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(tuple);
      return nullptr;
    }
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

// f with its refusals, and torch's errors, as Python's.
template <int ARGS, typename F>
PyObject* call(Py_ssize_t n, F f) noexcept {
  HANDLE_TH_ERRORS
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// logits, u, temperature, top_k, top_p, min_p
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<6>(n_args, [&] {
    const at::Tensor& logits = tensor(a[0], "logits");
    const int code = first(logits);
    two_dims(logits, "logits", "(rows, n)");
    const int64_t rows = logits.size(0), n = logits.size(1), ld = matrix(logits, rows, n, "logits");
    const at::Device device = logits.device();
    const float* u = vector<float>(a[1], at::kFloat, device, rows, "u");
    double temperature, top_k, top_p, min_p;
    const float* temperatures = by_row<float>(a[2], at::kFloat, device, rows, "temperature", &temperature);
    const int32_t* top_ks = by_row<int32_t>(a[3], at::kInt, device, rows, "top_k", &top_k);
    const float* top_ps = by_row<float>(a[4], at::kFloat, device, rows, "top_p", &top_p);
    const float* min_ps = by_row<float>(a[5], at::kFloat, device, rows, "min_p", &min_p);
    const int64_t k = top_ks ? 0 : whole(a[3], "top_k");
    Launch launch(device);
    const at::Tensor tokens = empty({rows}, at::kLong, device), logprobs = empty({rows}, at::kFloat, device);
    const int status = topk_sample(logits.data_ptr(), ld, code, rows, n, u, temperature, temperatures, k, top_ks, top_p, top_ps, min_p, min_ps,
                            static_cast<int64_t*>(tokens.data_ptr()), static_cast<float*>(logprobs.data_ptr()), stream_of(device));
    launch.done();
    return give(status, {tokens, logprobs});
  });
}

// x, idx, experts
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<3>(n_args, [&] {
    const at::Tensor& x = tensor(a[0], "x");
    const int code = first(x);
    two_dims(x, "x", "(tokens, d)");
    const int64_t tokens = x.size(0), d = x.size(1), ldx = matrix(x, tokens, d, "x"), experts = whole(a[2], "experts");
    const at::Device device = x.device();
    const at::Tensor& idx = choices(a[1], tokens, device, "idx");
    const int64_t k = idx.size(1);
    Launch launch(device);
    const at::Tensor xs = empty({tokens * k, d}, x.scalar_type(), device), place = empty({tokens, k}, at::kLong, device),
                     offsets = empty({experts < 0 || experts > (1 << 20) ? 1 : experts + 1}, at::kLong, device);
    const int status = topk_dispatch(x.data_ptr(), ldx, static_cast<const int64_t*>(idx.data_ptr()), code, tokens, k, experts, d, xs.data_ptr(),
                              static_cast<int64_t*>(place.data_ptr()), static_cast<int64_t*>(offsets.data_ptr()), stream_of(device));
    launch.done();
    return give(status, {xs, place, offsets});
  });
}

// ys, place, weights
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<3>(n_args, [&] {
    const at::Tensor& ys = tensor(a[0], "ys");
    const int code = first(ys);
    two_dims(ys, "ys", "(rows, d)");
    const int64_t rows = ys.size(0), d = ys.size(1), ldys = matrix(ys, rows, d, "ys");
    const at::Device device = ys.device();
    const at::Tensor& place = choices(a[1], -1, device, "place");
    const void* weights = of_places(a[2], place, ys.scalar_type(), device, "weights");
    const int64_t tokens = place.size(0);
    Launch launch(device);
    const at::Tensor y = empty({tokens, d}, ys.scalar_type(), device);
    const int status = topk_combine(ys.data_ptr(), ldys, rows, static_cast<const int64_t*>(place.data_ptr()), weights, code, tokens, place.size(1),
                             d, y.data_ptr(), stream_of(device));
    launch.done();
    return give(status, {y});
  });
}

// dy, ys, place, weights, whether dys is wanted, whether dweights is
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<6>(n_args, [&]() -> PyObject* {
    const at::Tensor& dy = tensor(a[0], "dy");
    const int code = first(dy);
    two_dims(dy, "dy", "(tokens, d)");
    const int64_t tokens = dy.size(0), d = dy.size(1);
    const at::Device device = dy.device();
    const at::Tensor& ys = like(a[1], dy.scalar_type(), device, "ys");
    two_dims(ys, "ys", "(rows, d)");
    const int64_t rows = ys.size(0), lddy = matrix(dy, tokens, d, "dy"), ldys = matrix(ys, rows, d, "ys");
    const at::Tensor& place = choices(a[2], tokens, device, "place");
    const void* weights = of_places(a[3], place, dy.scalar_type(), device, "weights");
    const int64_t k = place.size(1);
    const int want_dys = PyObject_IsTrue(a[4]), want_dweights = want_dys < 0 ? -1 : PyObject_IsTrue(a[5]);
    if (want_dweights < 0) return nullptr;
    Launch launch(device);
    at::Tensor dys, dweights;
    if (want_dys) dys = empty({rows, d}, dy.scalar_type(), device);
    if (want_dweights) dweights = empty({tokens, k}, dy.scalar_type(), device);
    const int status = topk_combine_backward(dy.data_ptr(), lddy, ys.data_ptr(), ldys, rows, static_cast<const int64_t*>(place.data_ptr()), weights,
                                      code, tokens, k, d, dys.defined() ? dys.data_ptr() : nullptr,
                                      dweights.defined() ? dweights.data_ptr() : nullptr, stream_of(device));
    launch.done();
    return give(status, {dys, dweights});
  });
}

// What evict and replace_ have in common.
struct Cache {
  int code, weights_code;
  int64_t batch, heads, capacity, key_dim, value_dim, group = 1, queries = 0;
  topk_view_t keys, values, score, weights{};
  const int64_t* lengths;
  bool weighted;
};
Cache cache_of(const at::Tensor& keys, PyObject* values_, PyObject* score_, PyObject* lengths_, PyObject* weights_) {
  Cache c;
  c.code = c.weights_code = first(keys);
  if (keys.dim() != 4) refuse(PyExc_ValueError, "keys must be 4-D (batch, heads, capacity, dim)");
  c.batch = keys.size(0), c.heads = keys.size(1), c.capacity = keys.size(2), c.key_dim = keys.size(3);
  const at::Device device = keys.device();
  const at::Tensor& values = like(values_, keys.scalar_type(), device, "values");
  if (values.dim() != 4) refuse(PyExc_ValueError, "values must be 4-D (batch, heads, capacity, dim)");
  c.value_dim = values.size(3);
  c.keys = view(keys, keys.sizes(), "keys");
  c.values = view(values, {c.batch, c.heads, c.capacity, c.value_dim}, "values");
  c.score = view(like(score_, at::kFloat, device, "score"), {c.batch, c.heads, c.capacity}, "score");
  c.lengths = vector<int64_t>(lengths_, at::kLong, device, c.batch, "lengths");
  c.weighted = weights_ != Py_None;
  if (c.weighted) {
    const at::Tensor& w = tensor(weights_, "weights");
    if (w.device() != device || w.dim() != 4)
      refuse(PyExc_TypeError, "weights must be a 4-D float32 or bfloat16 tensor (batch, query heads, queries, capacity) on %s", device.str().c_str());
    c.weights_code = code_of(w);
    const int64_t query_heads = w.size(1);
    if (c.heads < 1 || query_heads < c.heads || query_heads % c.heads)
      refuse(PyExc_ValueError, "weights must have a multiple of the cache's %lld heads, got %lld", static_cast<long long>(c.heads),
             static_cast<long long>(query_heads));
    c.group = query_heads / c.heads;
    c.queries = w.size(2);
    c.weights = view(w, {c.batch, query_heads, c.queries, c.capacity}, "weights");
  }
  return c;
}

// keys, values, score, lengths, keep, recent, weights
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<7>(n_args, [&] {
    const at::Tensor& keys = tensor(a[0], "keys");
    const Cache c = cache_of(keys, a[1], a[2], a[3], a[6]);
    const int64_t keep = whole(a[4], "keep"), recent = whole(a[5], "recent"), rows = keep < 0 || keep > (int64_t(1) << 31) ? 0 : keep;
    const at::Device device = keys.device();
    const at::ScalarType dtype = keys.scalar_type();
    Launch launch(device);
    const at::Tensor out_keys = empty({c.batch, c.heads, rows, c.key_dim}, dtype, device), out_values = empty({c.batch, c.heads, rows, c.value_dim}, dtype, device),
                     score = empty({c.batch, c.heads, rows}, at::kFloat, device), kept = empty({c.batch, c.heads, rows}, at::kLong, device),
                     lengths = empty({c.batch}, at::kLong, device);
    const int status = topk_evict(&c.keys, &c.values, &c.score, c.lengths, c.weighted ? &c.weights : nullptr, c.weights_code, c.group, c.queries, c.code,
                           c.batch, c.heads, c.capacity, c.key_dim, c.value_dim, keep, recent, out_keys.data_ptr(), out_values.data_ptr(),
                           static_cast<float*>(score.data_ptr()), static_cast<int64_t*>(kept.data_ptr()),
                           static_cast<int64_t*>(lengths.data_ptr()), stream_of(device));
    launch.done();
    return give(status, {out_keys, out_values, score, kept, lengths});
  });
}

// Tells autograd that t was written to, as torch's in-place operators do: a backward pass that saved it before raises an error
// instead of reading the new values.  (Tensors of inference mode keep no count.)
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// keys, values, score, positions, lengths, key, value, recent, weights
PyObject* replace(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return call<9>(n_args, [&] {
    const at::Tensor& keys = tensor(a[0], "keys");
    const Cache c = cache_of(keys, a[1], a[2], a[4], a[8]);
    const at::Device device = keys.device();
    const at::ScalarType dtype = keys.scalar_type();
    const topk_view_t positions = view(like(a[3], at::kLong, device, "positions"), {c.batch, c.heads, c.capacity}, "positions");
    const topk_view_t key = view(like(a[5], dtype, device, "key"), {c.batch, c.heads, c.key_dim}, "key");
    const topk_view_t value = view(like(a[6], dtype, device, "value"), {c.batch, c.heads, c.value_dim}, "value");
    const int64_t recent = whole(a[7], "recent");
    Launch launch(device);
    const at::Tensor slots = empty({c.batch, c.heads}, at::kLong, device);
    const int status = topk_replace(&c.keys, &c.values, &c.score, &positions, c.lengths, &key, &value, c.weighted ? &c.weights : nullptr,
                             c.weights_code, c.group, c.queries, c.code, c.batch, c.heads, c.capacity, c.key_dim, c.value_dim, recent,
                             static_cast<int64_t*>(slots.data_ptr()), stream_of(device));
    launch.done();
    if (status == TOPK_OK)
      for (int i = 0; i < 4; ++i) changed(tensor(a[i], ""));
    return give(status, {slots});
  });
}

template <typename F>
PyMethodDef method(const char* name, F f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("sample", sample),   method("dispatch", dispatch), method("combine", combine), method("combine_backward", combine_backward),
                         method("evict", evict),     method("replace", replace),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_language_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__language_calls() { return PyModule_Create(&module); }
