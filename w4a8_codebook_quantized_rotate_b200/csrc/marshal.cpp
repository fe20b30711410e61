// Python calls of the 8-bit integer path (include/w4a8_int8.h) on torch
// tensors: argument checks, output tensors, the current stream, and the C
// call.  The short calls of a decode step take 3 to 12 us on the GPU; checked
// and packed in Python they took 12 to 25 us of the host.
//
// Positional arguments only; binding.py gives them names, defaults and
// documentation.  Tensors must be contiguous, of the stated type and shape and
// on the current CUDA device (ValueError otherwise); a status of the library
// other than W4A8_OK raises binding.W4A8Error.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <optional>
#include <stdexcept>
#include <string>

#include "w4a8_int8.h"

namespace {

PyObject* g_error = nullptr;  // binding.W4A8Error
PyObject* g_cache_names[4];   // attributes of a cache: codes and scales of K and V

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused(what); }

const at::Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = optional(o, name);
  if (!t) refuse(std::string(name) + " must be a tensor");
  return *t;
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void on_cuda(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
}
// The current device, for a call whose first tensor this is.
int device_for(const at::Tensor& t, const char* name) {
  on_cuda(t, name);
  return int(c10::cuda::current_device());
}
void on_device(const at::Tensor& t, int dev, const char* name) {
  on_cuda(t, name);
  if (t.get_device() != dev)
    refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", not on the current device cuda:" +
           std::to_string(dev));
}

// The address of a contiguous tensor of that type, and shape where one is given.
void* address(const at::Tensor& t, at::ScalarType type, int dev, const char* name, at::IntArrayRef shape = {}) {
  on_device(t, dev, name);
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  if (!shape.empty() && t.sizes() != shape) refuse(std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  return t.data_ptr();
}
template <typename T>
T* address(PyObject* o, at::ScalarType type, int dev, const char* name, at::IntArrayRef shape = {}) {
  const at::Tensor* t = optional(o, name);
  return t ? static_cast<T*>(address(*t, type, dev, name, shape)) : nullptr;
}
void dims(const at::Tensor& t, int64_t n, const char* name, const char* what) {
  if (t.dim() != n) refuse(std::string(name) + " must be " + what);
}

// Numbers are read before anything is launched (a refusal leaves Python's own error).
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) refuse("not a number");
  return float(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) refuse("not a truth value");
  return v != 0;
}

// The stream of a call, made the current one while the call runs: outputs and
// scratch that the call allocates then belong to it, and are not handed to
// another tensor before its work is done.
struct OnStream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  void* stream;
  OnStream(PyObject* o, int dev) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
      return;
    }
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) PyErr_Clear(), refuse("stream must be a CUDA stream");
    stream = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) PyErr_Clear(), refuse("stream must be a CUDA stream");
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), c10::DeviceIndex(dev)));
  }
};

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int dev) {
  // (past the dispatcher, which costs as much again as the allocation)
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, c10::DeviceIndex(dev)), std::nullopt);
}

// bf16 rows [tokens, heads, dim], the values of a head contiguous.
w4a8_heads heads(const at::Tensor& t, int dev, const char* name, int64_t tokens, int64_t dim) {
  on_device(t, dev, name);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3) refuse(std::string(name) + " must be a bf16 tensor [tokens, heads, D]");
  if (t.size(0) != tokens || t.size(2) != dim)
    refuse(std::string(name) + " must be [" + std::to_string(tokens) + ", heads, " + std::to_string(dim) + "], got " + text(t.sizes()));
  if (t.stride(2) != 1) refuse(std::string(name) + ": the values of a head must be contiguous");
  if (t.size(1) > INT32_MAX) refuse(std::string(name) + " has too many heads");
  // a dimension of one row has no stride of its own
  const int64_t head = t.size(1) == 1 ? dim : t.stride(1), token = tokens == 1 ? t.size(1) * dim : t.stride(0);
  return w4a8_heads{static_cast<uint16_t*>(t.data_ptr()), token, head, int32_t(t.size(1))};
}
const w4a8_heads kNone{nullptr, 0, 0, 0};

// The output of rows shaped like `like`: the one given, or a new tensor.
at::Tensor out_like(PyObject* given, const at::Tensor& like, int dev, const char* name) {
  const at::Tensor* t = optional(given, name);
  return t ? *t : make(like.sizes(), at::kBFloat16, dev);
}

w4a8_rope rope(PyObject* inv_freq, PyObject* interleaved, PyObject* factor, int dev) {
  w4a8_rope r{nullptr, 0, truth(interleaved), number(factor)};
  if (const at::Tensor* t = optional(inv_freq, "inv_freq")) {
    dims(*t, 1, "inv_freq", "[rot_dim / 2]");
    r.inv_freq = static_cast<const double*>(address(*t, at::kDouble, dev, "inv_freq"));
    if (t->size(0) > 4096) refuse("inv_freq is too long");
    r.rot_dim = int32_t(2 * t->size(0));
  }
  return r;
}

// A cache's tensors, as they are at this call.
w4a8_kv_cache cache_of(PyObject* cache, int dev) {
  static const char* const names[4] = {"k_codes", "v_codes", "k_scales", "v_scales"};
  w4a8_kv_cache c{};
  void* at[4];
  int64_t shape[4] = {0, 0, 0, 0};
  for (int i = 0; i < 4; ++i) {
    PyObject* o = PyObject_GetAttr(cache, g_cache_names[i]);
    if (!o) PyErr_Clear(), refuse("cache must be a KvCache");
    const at::Tensor t = THPVariable_Check(o) ? THPVariable_Unpack(o) : at::Tensor();
    Py_DECREF(o);
    if (!t.defined()) refuse("cache must be a KvCache");
    if (i == 0) {
      dims(t, 4, names[i], "[pages, kv_heads, page, D]");
      for (int d = 0; d < 4; ++d) shape[d] = t.size(d);
    }
    at[i] = address(t, i < 2 ? at::kChar : at::kFloat, dev, names[i], at::IntArrayRef(shape, i < 2 ? 4 : 2));
  }
  if (shape[1] > INT32_MAX || shape[2] > INT32_MAX || shape[3] > INT32_MAX) refuse("the cache is too large");
  c.k_codes = static_cast<int8_t*>(at[0]);
  c.v_codes = static_cast<int8_t*>(at[1]);
  c.k_scales = static_cast<float*>(at[2]);
  c.v_scales = static_cast<float*>(at[3]);
  c.pages = shape[0];
  c.kv_heads = int32_t(shape[1]);
  c.page = int32_t(shape[2]);
  c.head_dim = int32_t(shape[3]);
  return c;
}

w4a8_kv_batch batch_of(PyObject* table, PyObject* q_start, PyObject* kv_len, int64_t tokens, int dev) {
  const at::Tensor& t = tensor(table, "block_table");
  dims(t, 2, "block_table", "[batch, pages]");
  const int64_t b = t.size(0);
  w4a8_kv_batch r;
  r.table = static_cast<const int32_t*>(address(t, at::kInt, dev, "block_table"));
  r.table_stride = t.size(1);
  r.q_start = static_cast<const int32_t*>(address(tensor(q_start, "q_start"), at::kInt, dev, "q_start", {b + 1}));
  r.kv_len = static_cast<const int32_t*>(address(tensor(kv_len, "kv_len"), at::kInt, dev, "kv_len", {b}));
  r.batch = b;
  r.tokens = tokens;
  return r;
}

bool failed(const char* call, w4a8_status status) {
  if (status == W4A8_OK) return false;
  if (PyObject* e = PyObject_CallFunction(g_error, "si", call, int(status))) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return true;
}

// Runs a call's body: a refusal becomes a ValueError, any other C++ exception
// a RuntimeError, an error that Python holds stays.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    PyObject* r = body();
    if (r && PyErr_Occurred()) {  // a number that was none
      Py_DECREF(r);
      return nullptr;
    }
    return r;
  } catch (const Refused& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* int8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, rotate, stream
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor& x = tensor(a[0], "x");
    const int dev = device_for(x, "x");
    const bool f32 = x.scalar_type() == at::kFloat;
    if (!f32 && x.scalar_type() != at::kBFloat16) refuse("x must be bf16 or fp32");
    const void* xp = address(x, x.scalar_type(), dev, "x");
    dims(x, 2, "x", "[R, K]");
    const OnStream on(a[2], dev);
    at::Tensor codes = make(x.sizes(), at::kChar, dev), s = make({x.size(0)}, at::kFloat, dev);
    if (failed("w4a8_int8_quantize", w4a8_int8_quantize(xp, f32, x.size(0), x.size(1), truth(a[1]),
                                                        static_cast<int8_t*>(codes.data_ptr()),
                                                        static_cast<float*>(s.data_ptr()), on.stream)))
      return nullptr;
    return Py_BuildValue("NN", THPVariable_Wrap(codes), THPVariable_Wrap(s));
  });
}

PyObject* int8_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x_q, s_x, w_q, s_w, out, stream
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x_q"), &w = tensor(a[2], "w_q");
    dims(x, 2, "x_q", "[M, K]");
    dims(w, 2, "w_q", "[N, K]");
    const int dev = device_for(x, "x_q");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const auto* xp = static_cast<const int8_t*>(address(x, at::kChar, dev, "x_q"));
    const auto* wp = static_cast<const int8_t*>(address(w, at::kChar, dev, "w_q", {N, K}));
    const auto* sx = static_cast<const float*>(address(tensor(a[1], "s_x"), at::kFloat, dev, "s_x", {M}));
    const auto* sw = static_cast<const float*>(address(tensor(a[3], "s_w"), at::kFloat, dev, "s_w", {N}));
    const OnStream on(a[5], dev);
    const at::Tensor* given = optional(a[4], "out");
    at::Tensor out = given ? *given : make({M, N}, at::kBFloat16, dev);
    auto* y = static_cast<uint16_t*>(address(out, at::kBFloat16, dev, "out", {M, N}));
    if (failed("w4a8_int8_gemm", w4a8_int8_gemm(xp, sx, M, wp, sw, N, K, y, on.stream))) return nullptr;
    return THPVariable_Wrap(out);
  });
}

PyObject* int8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, w_q, s_w, rotate, workspace, out, stream
  return guarded(n, 7, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w_q");
    dims(x, 2, "x", "[M, K]");
    dims(w, 2, "w_q", "[N, K]");
    const int dev = device_for(x, "x");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0);
    const auto* xp = static_cast<const uint16_t*>(address(x, at::kBFloat16, dev, "x"));
    const auto* wp = static_cast<const int8_t*>(address(w, at::kChar, dev, "w_q", {N, K}));
    const auto* sw = static_cast<const float*>(address(tensor(a[2], "s_w"), at::kFloat, dev, "s_w", {N}));
    const bool rotate = truth(a[3]);
    const OnStream on(a[6], dev);
    const at::Tensor* ws = optional(a[4], "workspace");
    at::Tensor scratch;
    if (!ws) {
      const size_t need = w4a8_int8_linear_workspace_bytes(M, K, N);
      if (need == 0) {
        failed("w4a8_int8_linear_workspace_bytes", W4A8_ERR_SHAPE);
        return nullptr;
      }
      scratch = make({int64_t(need)}, at::kByte, dev);
      ws = &scratch;
    }
    const at::Tensor* given = optional(a[5], "out");
    at::Tensor out = given ? *given : make({M, N}, at::kBFloat16, dev);
    auto* y = static_cast<uint16_t*>(address(out, at::kBFloat16, dev, "out", {M, N}));
    if (failed("w4a8_int8_linear",
               w4a8_int8_linear(xp, M, K, rotate, wp, sw, N, y, address(*ws, at::kByte, dev, "workspace"),
                                size_t(ws->numel()), on.stream)))
      return nullptr;
    return THPVariable_Wrap(out);
  });
}

// q, k, positions, q_weight, k_weight, eps, inv_freq, interleaved, factor, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor *q = optional(a[0], "q"), *k = optional(a[1], "k");
    const at::Tensor* some = q ? q : k;
    if (!some) refuse("q or k is needed");
    dims(*some, 3, q ? "q" : "k", "[tokens, heads, D]");
    const int dev = device_for(*some, q ? "q" : "k");
    const int64_t T = some->size(0), D = some->size(2);
    if (D > 65536) refuse("heads of " + std::to_string(D) + " values");
    const OnStream on(a[11], dev);
    const float eps = number(a[5]);
    w4a8_heads qs = kNone, qo = kNone, ks = kNone, ko = kNone;
    at::Tensor q_out, k_out;
    if (q) {
      qs = heads(*q, dev, "q", T, D);
      q_out = out_like(a[9], *q, dev, "q_out");
      qo = heads(q_out, dev, "q_out", T, D);
    }
    if (k) {
      ks = heads(*k, dev, "k", T, D);
      k_out = out_like(a[10], *k, dev, "k_out");
      ko = heads(k_out, dev, "k_out", T, D);
    }
    const w4a8_rope r = rope(a[6], a[7], a[8], dev);
    if (failed("w4a8_qk_norm_rope",
               w4a8_qk_norm_rope(&qs, &ks, T, int32_t(D), address<const float>(a[3], at::kFloat, dev, "q_weight", {D}),
                                 address<const float>(a[4], at::kFloat, dev, "k_weight", {D}), eps,
                                 address<const int32_t>(a[2], at::kInt, dev, "positions", {T}), &r, &qo, &ko, on.stream)))
      return nullptr;
    return Py_BuildValue("NN", q ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None), k ? THPVariable_Wrap(k_out) : Py_NewRef(Py_None));
  });
}

// cache, k, v, block_table, q_start, kv_len, q, positions, q_weight, k_weight, eps, inv_freq, interleaved, factor, q_out,
// stream
PyObject* kv_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int dev = device_for(k, "k");
    const w4a8_kv_cache cache = cache_of(a[0], dev);
    const at::Tensor* q = optional(a[6], "q");
    dims(k, 3, "k", "[tokens, heads, D]");
    const int64_t T = k.size(0), D = cache.head_dim;
    const w4a8_kv_batch batch = batch_of(a[3], a[4], a[5], T, dev);
    const w4a8_heads ks = heads(k, dev, "k", T, D), vs = heads(v, dev, "v", T, D);
    const OnStream on(a[15], dev);
    w4a8_heads qs = kNone, qo = kNone;
    at::Tensor q_out;
    if (q) {
      qs = heads(*q, dev, "q", T, D);
      q_out = out_like(a[14], *q, dev, "q_out");
      qo = heads(q_out, dev, "q_out", T, D);
    }
    const w4a8_rope r = rope(a[11], a[12], a[13], dev);
    const float eps = number(a[10]);
    if (failed("w4a8_kv_update",
               w4a8_kv_update(&cache, &batch, &ks, &vs, &qs, address<const float>(a[8], at::kFloat, dev, "q_weight", {D}),
                              address<const float>(a[9], at::kFloat, dev, "k_weight", {D}), eps,
                              address<const int32_t>(a[7], at::kInt, dev, "positions", {T}), &r, &qo, on.stream)))
      return nullptr;
    return q ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
  });
}

PyObject* kv_dequant(PyObject*, PyObject* const* a, Py_ssize_t n) {  // cache, ids, stream
  return guarded(n, 3, [&]() -> PyObject* {
    const at::Tensor& ids = tensor(a[1], "ids");
    const int dev = device_for(ids, "ids");
    const w4a8_kv_cache cache = cache_of(a[0], dev);
    dims(ids, 1, "ids", "[n]");
    const auto* at = static_cast<const int32_t*>(address(ids, at::kInt, dev, "ids"));
    const int64_t shape[4] = {ids.size(0), cache.kv_heads, cache.page, cache.head_dim};
    const OnStream on(a[2], dev);
    at::Tensor k = make(shape, at::kBFloat16, dev), v = make(shape, at::kBFloat16, dev);
    if (failed("w4a8_kv_dequant", w4a8_kv_dequant(&cache, at, ids.size(0), static_cast<uint16_t*>(k.data_ptr()),
                                                  static_cast<uint16_t*>(v.data_ptr()), on.stream)))
      return nullptr;
    return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
  });
}

// q, cache, block_table, q_start, kv_len, scale (None: D ** -0.5), window, workspace, out, stream
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const int dev = device_for(q, "q");
    dims(q, 3, "q", "[tokens, heads, D]");
    const w4a8_kv_cache cache = cache_of(a[1], dev);
    const int64_t T = q.size(0), D = cache.head_dim;
    const w4a8_heads qs = heads(q, dev, "q", T, D);
    const w4a8_kv_batch batch = batch_of(a[2], a[3], a[4], T, dev);
    const float scale = a[5] == Py_None ? 1.f / std::sqrt(float(D)) : number(a[5]);
    const long window = PyLong_AsLong(a[6]);
    if (window < 0 || window > INT32_MAX) refuse("window must be a whole number of tokens");
    const OnStream on(a[9], dev);
    const at::Tensor* ws = optional(a[7], "workspace");
    at::Tensor scratch;
    if (!ws) {
      const size_t need = w4a8_kv_attention_workspace_bytes(T, qs.heads, cache.kv_heads, cache.head_dim);
      if (need == 0) {
        failed("w4a8_kv_attention_workspace_bytes", W4A8_ERR_SHAPE);
        return nullptr;
      }
      scratch = at::zeros({int64_t(need)}, at::TensorOptions().dtype(at::kByte).device(at::Device(at::kCUDA, c10::DeviceIndex(dev))));
      ws = &scratch;
    }
    at::Tensor out = out_like(a[8], q, dev, "out");
    const w4a8_heads os = heads(out, dev, "out", T, D);
    if (failed("w4a8_kv_attention", w4a8_kv_attention(&qs, &cache, &batch, scale, int32_t(window), &os,
                                                      address(*ws, at::kByte, dev, "workspace"), size_t(ws->numel()), on.stream)))
      return nullptr;
    return THPVariable_Wrap(out);
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

#define CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {CALL(int8_quantize), CALL(int8_gemm),  CALL(int8_linear),  CALL(qk_norm_rope),
                          CALL(kv_update),     CALL(kv_dequant), CALL(kv_attention), {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "w4a8_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_w4a8_marshal() {
  const char* const names[4] = {"k_codes", "v_codes", "k_scales", "v_scales"};
  for (int i = 0; i < 4; ++i)
    if (!(g_cache_names[i] = PyUnicode_InternFromString(names[i]))) return nullptr;
  return PyModule_Create(&kModule);
}
