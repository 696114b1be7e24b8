// torch_calls.cpp — Python module _torch_calls: the routing, combine and int8 calls of
// include/moe.h on torch tensors (the documented entry points are in routed.py, int8.py).
//
// These calls are a few microseconds of GPU work each when batches are small, so what the
// host spends on checks and marshalling is their time: in Python, over ctypes, 4 to 9 us a
// call; here about 1. Every tensor is checked (type, shape, device, contiguous) before the
// library is called; the library checks the rest. The work goes to the current stream of
// the tensors' device, which need not be the current device.
//
// The module calls the library through the addresses that setup() is given, so that it
// serves whichever build of it is loaded.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstdint>
#include <initializer_list>
#include <limits>
#include <optional>
#include <string>

#include "moe.h"

namespace {

struct Library {
  decltype(&moe_topk_workspace_size) topk_workspace_size = nullptr;
  decltype(&moe_topk_route) topk_route = nullptr;
  decltype(&moe_topk_route_backward) topk_route_backward = nullptr;
  decltype(&moe_combine_topk) combine_topk = nullptr;
  decltype(&moe_int8_workspace_size) int8_workspace_size = nullptr;
  decltype(&moe_int8_product) int8_product = nullptr;
} lib;
PyObject* moe_error = nullptr;  // class MoeError(status, what)

// A Python exception is set.
struct Raised {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, ("moe: " + what).c_str());
  throw Raised();
}

std::string shape_of(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor, not " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// The tensor that the others are held against.
const at::Tensor& first(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) refuse(std::string(name) + " must live on a CUDA device");
  if (t.dim() != dims)
    refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions, not " + std::to_string(t.dim()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t;
}

const at::Tensor& need(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.device() != dev)
    refuse(std::string(name) + " is on " + t.device().str() + ", the call's other tensors on " + dev.str());
  if (t.scalar_type() != type)
    refuse(std::string(name) + " has type " + c10::toString(t.scalar_type()) + ", not " + c10::toString(type));
  if (t.sizes() != shape) refuse(std::string(name) + " has shape " + shape_of(t.sizes()) + ", not " + shape_of(shape));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  return t;
}

// Address of an input that may be None.
template <typename T>
const T* input(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return o == Py_None ? nullptr : static_cast<const T*>(need(o, name, shape, type, dev).const_data_ptr());
}

moe_dtype_t code(at::ScalarType type, const char* name) {
  if (type == at::kFloat) return MOE_F32;
  if (type == at::kBFloat16) return MOE_BF16;
  refuse(std::string(name) + " has type " + c10::toString(type) + ", not fp32 or bf16");
}

int32_t int32_of(int64_t v, const char* name) {
  if (v < std::numeric_limits<int32_t>::min() || v > std::numeric_limits<int32_t>::max())
    refuse(std::string(name) + " is out of range");
  return static_cast<int32_t>(v);
}

int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return int32_of(v, name);
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

at::ScalarType type_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse("out_dtype must be a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// Uint8 workspace: the caller's (whatever its size: the library says if it is too small), or
// one of `size` bytes that lives until the call is on its stream.
struct Workspace {
  at::Tensor held;
  void* at = nullptr;
  size_t bytes = 0;

  Workspace(PyObject* given, size_t size, at::Device dev) {
    if (given != Py_None) {
      const at::Tensor& t = tensor(given, "workspace");
      need(given, "workspace", {t.numel()}, at::kByte, dev);
      held = t;
    } else if (size > 0) {
      held = empty({static_cast<int64_t>(size)}, at::kByte, dev);
    } else {
      return;
    }
    at = held.mutable_data_ptr();
    bytes = static_cast<size_t>(held.numel());
  }
};

// Runs the library's call with the tensors' device current, on its current stream.
template <typename F>
void launch(const char* what, F call) {
  moe_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = call();
  Py_END_ALLOW_THREADS
  if (st == MOE_OK) return;
  PyObject* e = PyObject_CallFunction(moe_error, "is", static_cast<int>(st), what);
  if (e != nullptr) {
    PyErr_SetObject(moe_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

void* stream_of(at::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// A result: the caller's tensor, or a new one.
struct Result {
  PyObject* object = nullptr;  // owned
  void* at = nullptr;
  at::ScalarType type;

  Result(PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType t, at::Device dev, bool zeros = false)
      : type(t) {
    if (given != nullptr && given != Py_None) {
      const at::Tensor& out = need(given, name, shape, t, dev);
      at = out.mutable_data_ptr();
      // what autograd has saved of it is no longer what it was
      if (!out.is_inference()) out.unsafeGetTensorImpl()->bump_version();
      object = Py_NewRef(given);
    } else {
      at::Tensor made = empty(shape, t, dev);
      if (zeros) made.zero_();
      at = made.mutable_data_ptr();
      object = THPVariable_Wrap(std::move(made));
      if (object == nullptr) throw Raised();
    }
  }
  Result(const Result&) = delete;
  ~Result() { Py_XDECREF(object); }
  PyObject* release() {
    PyObject* o = object;
    object = nullptr;
    return o;
  }
};

// The type of an output that is given or not.
at::ScalarType out_type(PyObject* out, PyObject* dtype, at::ScalarType otherwise) {
  if (out == Py_None) return type_of(dtype, otherwise);
  const at::ScalarType t = tensor(out, "out").scalar_type();
  const at::ScalarType asked = type_of(dtype, t);
  if (asked != t) refuse(std::string("out has type ") + c10::toString(t) + ", not " + c10::toString(asked));
  return t;
}

moe_topk_args_t topk_args(const at::Tensor& logits, int32_t k, PyObject* score, PyObject* renorm, PyObject* scale,
                          PyObject* n_tokens) {
  moe_topk_args_t a{};
  a.logits = logits.const_data_ptr();
  a.T = logits.size(0);
  a.E = int32_of(logits.size(1), "the number of experts");
  a.k = k;
  a.dtype = code(logits.scalar_type(), "logits");
  a.score = static_cast<moe_score_t>(integer(score, "score"));
  a.renormalize = truth(renorm) ? 1 : 0;
  a.scale = number(scale);
  a.n_groups = a.topk_groups = 1;
  a.group_rule = MOE_GROUP_MAX;
  if (n_tokens != Py_None) {
    const at::Tensor& t = tensor(n_tokens, "n_tokens");
    if (t.numel() != 1) refuse("n_tokens must hold one number");
    a.n_tokens = input<int32_t>(n_tokens, "n_tokens", t.sizes(), at::kInt, logits.device());
  }
  return a;
}

// topk_route(logits, k, score, bias, n_groups, topk_groups, group_rule, renormalize, scale,
//            n_tokens, want_scores, dispatch, out, workspace) -> dict
constexpr int kNames = 9;
const char* const kName[kNames] = {"idx", "weights", "scores", "counts", "offsets", "perm_token", "perm_slot",
                                   "slot_pos", "gate_perm"};
PyObject* name_object[kNames];

PyObject* topk_route(PyObject* const* v) {
  const at::Tensor& logits = first(v[0], "logits", 2);
  const at::Device dev = logits.device();
  moe_topk_args_t a = topk_args(logits, integer(v[1], "k"), v[2], v[7], v[8], v[9]);
  a.bias = input<float>(v[3], "bias", {a.E}, at::kFloat, dev);
  a.n_groups = integer(v[4], "n_groups");
  a.topk_groups = integer(v[5], "topk_groups");
  a.group_rule = static_cast<moe_group_rule_t>(integer(v[6], "group_rule"));
  const bool want_scores = truth(v[10]), dispatch = truth(v[11]);
  PyObject* given = v[12] == Py_None ? nullptr : v[12];
  if (given != nullptr && !PyDict_Check(given)) refuse("out must be a dict");
  const int64_t T = a.T, E = a.E, n = a.k > 0 ? a.k : 0, slots = T * n;
  const c10::cuda::CUDAGuard guard(dev);
  struct Dict {
    PyObject* o = PyDict_New();
    ~Dict() { Py_XDECREF(o); }
  } res;
  if (res.o == nullptr) throw Raised();
  std::array<void*, kNames> at{};
  Py_ssize_t used = 0;
  auto put = [&](int i, at::IntArrayRef shape, at::ScalarType type) {
    PyObject* g = nullptr;
    if (given != nullptr) {
      g = PyDict_GetItemWithError(given, name_object[i]);
      if (g == nullptr && PyErr_Occurred()) throw Raised();
      used += g != nullptr;
    }
    Result r(g, kName[i], shape, type, dev);
    at[i] = r.at;
    if (PyDict_SetItem(res.o, name_object[i], r.object) < 0) throw Raised();
  };
  put(0, {T, n}, at::kInt);
  put(1, {T, n}, at::kFloat);
  if (want_scores) put(2, {T, E}, at::kFloat);
  if (dispatch) {
    put(3, {E}, at::kInt);
    put(4, {E + 1}, at::kInt);
    put(5, {slots}, at::kInt);
    put(6, {slots}, at::kInt);
    put(7, {T, n}, at::kInt);
    put(8, {slots}, at::kFloat);
  }
  if (given != nullptr && PyDict_Size(given) > used) refuse("out holds tensors that this call does not write");
  const Workspace ws(v[13], dispatch && v[13] == Py_None ? lib.topk_workspace_size(T, a.E, a.k) : 0, dev);
  const moe_topk_routed_t r{static_cast<int32_t*>(at[0]), static_cast<float*>(at[1]),   static_cast<float*>(at[2]),
                            static_cast<int32_t*>(at[3]), static_cast<int32_t*>(at[4]), static_cast<int32_t*>(at[5]),
                            static_cast<int32_t*>(at[6]), static_cast<int32_t*>(at[7]), static_cast<float*>(at[8])};
  void* const s = stream_of(dev);
  launch("moe_topk_route", [&] { return lib.topk_route(&a, &r, ws.at, ws.bytes, s); });
  return Py_NewRef(res.o);
}

// topk_route_backward(logits, idx, grad_weights, score, renormalize, scale, grad_scores, n_tokens, out)
PyObject* topk_route_backward(PyObject* const* v) {
  const at::Tensor& logits = first(v[0], "logits", 2);
  const at::Device dev = logits.device();
  const at::Tensor& idx = first(v[1], "idx", 2);
  const int64_t T = logits.size(0), k = idx.size(1);
  const moe_topk_args_t a = topk_args(logits, int32_of(k, "the number of choices"), v[3], v[4], v[5], v[7]);
  const int32_t* ip = input<int32_t>(v[1], "idx", {T, k}, at::kInt, dev);
  const float* gp = static_cast<const float*>(need(v[2], "grad_weights", {T, k}, at::kFloat, dev).const_data_ptr());
  const float* sp = input<float>(v[6], "grad_scores", logits.sizes(), at::kFloat, dev);
  const c10::cuda::CUDAGuard guard(dev);
  Result g(v[8], "out", logits.sizes(), logits.scalar_type(), dev);
  void* const s = stream_of(dev);
  launch("moe_topk_route_backward", [&] { return lib.topk_route_backward(&a, ip, gp, sp, g.at, s); });
  return g.release();
}

// combine_topk(y, slot_pos, weights, residual, out, out_dtype)
PyObject* combine_topk(PyObject* const* v) {
  const at::Tensor& y = first(v[0], "y", 2);
  const at::Device dev = y.device();
  const at::Tensor& pos = first(v[1], "slot_pos", 2);
  const int64_t R = y.size(0), d = y.size(1), T = pos.size(0), k = pos.size(1);
  const moe_dtype_t yc = code(y.scalar_type(), "y");
  const int32_t kc = int32_of(k, "the number of slots");
  const int32_t* pp = input<int32_t>(v[1], "slot_pos", {T, k}, at::kInt, dev);
  const float* wp = input<float>(v[2], "weights", {T, k}, at::kFloat, dev);
  const at::ScalarType type =
      out_type(v[4], v[5], v[3] == Py_None ? y.scalar_type() : tensor(v[3], "residual").scalar_type());
  const moe_dtype_t oc = code(type, "out");
  const void* rp = input<void>(v[3], "residual", {T, d}, type, dev);
  const c10::cuda::CUDAGuard guard(dev);
  Result o(v[4], "out", {T, d}, type, dev);
  const void* yp = y.const_data_ptr();
  void* const s = stream_of(dev);
  launch("moe_combine_topk", [&] { return lib.combine_topk(yp, yc, R, pp, wp, T, kc, d, rp, o.at, oc, s); });
  return o.release();
}

// int8_product(x, w, s, x_scale, index, counts, w_up, s_up, activation, gate, out, out_dtype, workspace)
PyObject* int8_product(PyObject* const* v) {
  const at::Tensor& x = first(v[0], "x", 2);
  const at::Device dev = x.device();
  const at::Tensor& w = first(v[1], "w", 3);
  moe_int8_args_t a{};
  a.x_rows = x.size(0);
  const int64_t n = w.size(0);
  a.K = w.size(1);
  a.N = w.size(2);
  a.n_experts = int32_of(n, "the number of experts");
  a.x_dtype = x.scalar_type() == at::kChar ? MOE_INT8 : code(x.scalar_type(), "x");
  if (x.size(1) != a.K)
    refuse("x has rows of " + std::to_string(x.size(1)) + ", w of " + std::to_string(a.K));
  a.R = v[4] == Py_None ? a.x_rows : tensor(v[4], "index").numel();
  if ((v[6] == Py_None) != (v[7] == Py_None)) refuse("w_up and s_up come together");
  a.x = x.const_data_ptr();
  a.x_scale = input<float>(v[3], "x_scale", {a.R}, at::kFloat, dev);
  a.index = input<int32_t>(v[4], "index", {a.R}, at::kInt, dev);
  a.counts = input<int32_t>(v[5], "counts", {n}, at::kInt, dev);
  a.w = need(v[1], "w", w.sizes(), at::kChar, dev).const_data_ptr();
  a.w_up = input<void>(v[6], "w_up", w.sizes(), at::kChar, dev);
  a.s = need(v[2], "s", {n, a.N}, at::kBFloat16, dev).const_data_ptr();
  a.s_up = input<void>(v[7], "s_up", {n, a.N}, at::kBFloat16, dev);
  a.gate = input<float>(v[9], "gate", {a.R}, at::kFloat, dev);
  a.activation = static_cast<moe_activation_t>(integer(v[8], "activation"));
  const at::ScalarType type = out_type(v[10], v[11], at::kBFloat16);
  a.out_dtype = code(type, "out");
  const c10::cuda::CUDAGuard guard(dev);
  Result o(v[10], "out", {a.R, a.N}, type, dev, a.counts != nullptr);
  a.out = o.at;
  const size_t size = v[12] == Py_None ? lib.int8_workspace_size(a.R, a.K, a.N, a.n_experts, a.x_dtype,
                                                                 a.w_up != nullptr ? 1 : 0)
                                       : 0;
  const Workspace ws(v[12], size, dev);
  void* const s = stream_of(dev);
  launch("moe_int8_product", [&] { return lib.int8_product(&a, ws.at, ws.bytes, s); });
  return o.release();
}

// setup(MoeError, addresses of the six functions in Library's order)
PyObject* setup(PyObject* const* v) {
  Py_XSETREF(moe_error, Py_NewRef(v[0]));
  void* at[6];
  for (int i = 0; i < 6; ++i) {
    at[i] = PyLong_AsVoidPtr(v[1 + i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "moe: no such function in the library");
      throw Raised();
    }
  }
  lib.topk_workspace_size = reinterpret_cast<decltype(lib.topk_workspace_size)>(at[0]);
  lib.topk_route = reinterpret_cast<decltype(lib.topk_route)>(at[1]);
  lib.topk_route_backward = reinterpret_cast<decltype(lib.topk_route_backward)>(at[2]);
  lib.combine_topk = reinterpret_cast<decltype(lib.combine_topk)>(at[3]);
  lib.int8_workspace_size = reinterpret_cast<decltype(lib.int8_workspace_size)>(at[4]);
  lib.int8_product = reinterpret_cast<decltype(lib.int8_product)>(at[5]);
  Py_RETURN_NONE;
}

// No C++ exception reaches the interpreter: torch's become its own Python errors.
template <PyObject* (*F)(PyObject* const*), int N, bool LIBRARY>
PyObject* entry(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    if (n != N) {
      PyErr_Format(PyExc_TypeError, "moe: %d arguments expected, %zd given", N, n);
      return nullptr;
    }
    if (LIBRARY && moe_error == nullptr) {
      PyErr_SetString(PyExc_RuntimeError, "moe: setup() has not been called");
      return nullptr;
    }
    return F(v);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N, bool LIBRARY = true>
PyCFunction as_function() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N, LIBRARY>));
}

PyMethodDef methods[] = {
    {"setup", as_function<setup, 7, false>(), METH_FASTCALL, nullptr},
    {"topk_route", as_function<topk_route, 14>(), METH_FASTCALL, nullptr},
    {"topk_route_backward", as_function<topk_route_backward, 9>(), METH_FASTCALL, nullptr},
    {"combine_topk", as_function<combine_topk, 6>(), METH_FASTCALL, nullptr},
    {"int8_product", as_function<int8_product, 13>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() {
  for (int i = 0; i < kNames; ++i)
    if (name_object[i] == nullptr && (name_object[i] = PyUnicode_InternFromString(kName[i])) == nullptr) return nullptr;
  return PyModule_Create(&module);
}
