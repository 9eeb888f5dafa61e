// Python entry of the operators around the layer (operators.py): checks of the tensors, the
// outputs' and workspaces' allocation, the current stream, and the call into the C ABI.
//
// The smallest of these calls are over on the GPU in a few microseconds; through ctypes,
// with the checks and allocations in Python, one took 14 us of the host (decode gate, of
// which the launch itself is 2).  So what happens once per call is compiled.
// Functions take their arguments by position, in the order of the comment above each.
//
// Errors: ValueError for a tensor that does not fit, QmoeError (handed over by
// operators.py) for a negative code of the library.  No C++ exception leaves a function
// (HANDLE_TH_ERRORS).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>
#include <sstream>
#include <string>

#include "qmoe.h"

namespace {

PyObject* g_error = nullptr;  // operators.py's QmoeError
PyObject* g_graph = nullptr;  // operators.py's _graph

// What a function throws to leave with a Python exception already set.
struct Raised {};

[[noreturn]] void fail(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Raised{};
}

[[noreturn]] void fail_shape(const char* name, std::initializer_list<int64_t> want,
                             at::IntArrayRef got) {
  std::ostringstream s;
  s << name << ": need shape (";
  const char* sep = "";
  for (int64_t w : want) {
    s << sep << w;
    sep = ", ";
  }
  s << "), got " << got;
  fail(s.str());
}

void check_rc(const char* fn, int rc) {
  if (rc == QMOE_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "si", fn, rc) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s failed (%d)", fn, rc);
  }
  throw Raised{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(std::string(name) + ": need a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}
// A size for the C ABI: out of int's range is out of every limit of the library too.
int small(int64_t v) { return v < -1 ? -1 : v > INT32_MAX ? INT32_MAX : (int)v; }

int dtype_code(at::ScalarType t) {
  if (t == at::kBFloat16) return QMOE_DTYPE_BF16;
  if (t == at::kHalf) return QMOE_DTYPE_FP16;
  return t == at::kFloat ? QMOE_DTYPE_FP32 : -1;
}

// Whether autograd has to know of a call on this argument.
bool needs_gradient(PyObject* o) {
  return o != Py_None && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad();
}
// The call `name` with n arguments again, from within a node of autograd's graph.
PyObject* in_graph(const char* name, PyObject* const* a, Py_ssize_t n) {
  PyObject* args = PyTuple_New(n + 1);
  if (!args) throw Raised{};
  PyObject* s = PyUnicode_FromString(name);
  if (!s) {
    Py_DECREF(args);
    throw Raised{};
  }
  PyTuple_SET_ITEM(args, 0, s);
  for (Py_ssize_t i = 0; i < n; ++i) {
    Py_INCREF(a[i]);
    PyTuple_SET_ITEM(args, i + 1, a[i]);
  }
  PyObject* r = PyObject_Call(g_graph, args, nullptr);
  Py_DECREF(args);
  if (!r) throw Raised{};
  return r;
}

// Operators whose default workspaces are kept.
enum Kept { kSort, kLora, kKeptKinds };
constexpr int kDevices = 64;

// The device of a call: every tensor has to be on the current one.
struct Call {
  c10::DeviceIndex dev = -1;
  void here(const at::Tensor& t, const char* name) {
    if (t.is_cuda()) {
      if (dev < 0) dev = c10::cuda::current_device();
      if (t.get_device() == dev) return;
    }
    fail(std::string(name) + ": need a tensor on the current CUDA device, got " +
         t.device().str());
  }
  // A matrix of activation rows: its row stride in elements (0: the same row throughout).
  long long rows(const at::Tensor& t, const char* name) {
    if (t.dim() != 2 || dtype_code(t.scalar_type()) < 0 || t.layout() != at::kStrided)
      fail(std::string(name) + ": need a matrix of bf16, fp16 or fp32");
    here(t, name);
    if (t.size(1) > 1 && t.stride(1) != 1)
      fail(std::string(name) + ": the elements of a row must be next to each other");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
  }
  long long rows(const at::Tensor& t, const char* name, int64_t n, int64_t width) {
    const long long ld = rows(t, name);
    if (t.size(0) != n || t.size(1) != width) fail_shape(name, {n, width}, t.sizes());
    return ld;
  }
  void dense(const at::Tensor& t, at::ScalarType type, const char* name,
             std::initializer_list<int64_t> shape) {
    if (t.scalar_type() != type || t.layout() != at::kStrided || !t.is_contiguous())
      fail(std::string(name) + ": need a contiguous tensor of " + c10::toString(type) + ", got " +
           c10::toString(t.scalar_type()));
    here(t, name);
    if (t.sizes() != at::IntArrayRef(shape.begin(), shape.size()))
      fail_shape(name, shape, t.sizes());
  }
  at::Tensor make(at::ScalarType type, std::initializer_list<int64_t> shape) {
    for (int64_t n : shape)
      if (n < 0) fail("a negative size");
    return at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), type,
                                  at::Device(at::kCUDA, dev), std::nullopt);
  }
  // A given output, or a new one.
  at::Tensor out(PyObject* o, at::ScalarType type, const char* name,
                 std::initializer_list<int64_t> shape) {
    if (o == Py_None) return make(type, shape);
    const at::Tensor& t = tensor(o, name);
    dense(t, type, name, shape);
    return t;
  }
  at::Tensor space(PyObject* o, size_t bytes, Kept which) {
    if (o == Py_None) {
      kept(which) = at::Tensor();  // its memory may serve again
      return make(at::kByte, {(int64_t)(bytes < 256 ? 256 : bytes)});
    }
    const at::Tensor& t = tensor(o, "workspace");
    dense(t, at::kByte, "workspace", {t.numel()});
    return t;
  }
  // The workspace of the last call that brought none, for its error word (one per operator
  // and device; never destroyed, since that could come after the CUDA context's end).
  at::Tensor& kept(Kept which) const {
    static auto* all = new std::array<at::Tensor, kDevices * kKeptKinds>();
    if (dev < 0 || dev >= kDevices) fail("too many CUDA devices");
    return (*all)[(size_t)(dev * kKeptKinds + which)];
  }
  // top_k of an [M][top_k] table
  int64_t slots(const at::Tensor& t, const char* name) {
    if (t.dim() != 2) fail(std::string(name) + ": need [M][top_k]");
    return t.size(1);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

const int32_t* i32(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }
int32_t* i32_out(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
float* f32(const at::Tensor& t) { return static_cast<float*>(t.data_ptr()); }

PyObject* pack(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F&& body) {
  HANDLE_TH_ERRORS
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return body();
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// logits, top_k, scoring, bias, n_group, topk_group, renormalize, scale, ids, weights
PyObject* gate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled() && needs_gradient(a[0]))
      return in_graph("gate", a, n);
    Call c;
    const at::Tensor& logits = tensor(a[0], "logits");
    const long long ld = c.rows(logits, "logits");
    const int64_t M = logits.size(0), E = logits.size(1), k = integer(a[1]);
    const float* bias = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& b = tensor(a[3], "bias");
      c.dense(b, at::kFloat, "bias", {E});
      bias = f32(b);
    }
    const double scale = PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) throw Raised{};
    if (k < 1 || k > 64) check_rc("moe_gate", QMOE_ERR_SHAPE);
    const at::Tensor ids = c.out(a[8], at::kInt, "topk_ids", {M, k});
    const at::Tensor w = c.out(a[9], at::kFloat, "topk_weights", {M, k});
    check_rc("moe_gate",
             moe_gate(logits.data_ptr(), dtype_code(logits.scalar_type()), ld, small(M), small(E),
                      (int)k, small(integer(a[2])), bias, small(integer(a[4])),
                      small(integer(a[5])), truth(a[6]), (float)scale, i32_out(ids),
                      f32(w), c.stream()));
    return pack({ids, w});
  });
}

// dweights, logits, ids, scoring, renormalize, scale, dlogits
PyObject* gate_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const at::Tensor& logits = tensor(a[1], "logits");
    const long long ld = c.rows(logits, "logits");
    const int64_t M = logits.size(0), E = logits.size(1);
    const at::Tensor& ids = tensor(a[2], "topk_ids");
    const int64_t k = c.slots(ids, "topk_ids");
    c.dense(ids, at::kInt, "topk_ids", {M, k});
    const at::Tensor& dw = tensor(a[0], "dweights");
    c.dense(dw, at::kFloat, "dweights", {M, k});
    const double scale = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) throw Raised{};
    const at::Tensor dl = c.out(a[6], logits.scalar_type(), "dlogits", {M, E});
    check_rc("moe_gate_backward",
             moe_gate_backward(f32(dw), logits.data_ptr(), dtype_code(logits.scalar_type()), ld,
                               i32(ids), small(M), small(E), small(k), small(integer(a[3])),
                               truth(a[4]), (float)scale, dl.data_ptr(), c.stream()));
    return THPVariable_Wrap(dl);
  });
}

// x, ids, E, xs, workspace
PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled() && needs_gradient(a[0]))
      return in_graph("sort_tokens", a, n);
    Call c;
    const at::Tensor& x = tensor(a[0], "x");
    const long long ldx = c.rows(x, "x");
    const int64_t M = x.size(0), H = x.size(1);
    const at::Tensor& ids = tensor(a[1], "topk_ids");
    const int64_t k = c.slots(ids, "topk_ids"), E = integer(a[2]);
    c.dense(ids, at::kInt, "topk_ids", {M, k});
    if (E < 1 || E > 2048) check_rc("moe_sort_tokens", QMOE_ERR_SHAPE);
    const at::Tensor xs = c.out(a[3], x.scalar_type(), "xs", {M * k, H});
    const at::Tensor offsets = c.make(at::kInt, {E + 1});
    if (M == 0) offsets.zero_();  // the call itself is a no-op then
    const at::Tensor pair = c.make(at::kInt, {M * k});
    const at::Tensor pos = c.make(at::kInt, {M, k});
    const at::Tensor ws =
        c.space(a[4], qmoe_sort_workspace_size(small(M), small(k), (int)E), kSort);
    check_rc("moe_sort_tokens",
             moe_sort_tokens(x.data_ptr(), dtype_code(x.scalar_type()), ldx, i32(ids), small(M),
                             small(H), small(k), (int)E, xs.data_ptr(), i32_out(offsets),
                             i32_out(pair), i32_out(pos), ws.data_ptr(), (size_t)ws.numel(),
                             c.stream()));
    if (a[4] == Py_None && M > 0) c.kept(kSort) = ws;  // (no tokens: no error word)
    return pack({xs, offsets, pair, pos});
  });
}

// dxs, pair_pos, dx
PyObject* sort_tokens_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    Call c;
    const at::Tensor& y = tensor(a[0], "dxs");
    const at::Tensor& pos = tensor(a[1], "pair_pos");
    const int64_t k = c.slots(pos, "pair_pos"), M = pos.size(0);
    c.dense(pos, at::kInt, "pair_pos", {M, k});
    const long long ld = c.rows(y, "dxs");
    const int64_t H = y.size(1);
    if (y.size(0) != M * k) fail_shape("dxs", {M * k, H}, y.sizes());
    const at::Tensor dx = c.out(a[2], y.scalar_type(), "dx", {M, H});
    check_rc("moe_sort_tokens_backward",
             moe_sort_tokens_backward(y.data_ptr(), dtype_code(y.scalar_type()), ld, i32(pos),
                                      small(M), small(H), small(k), dx.data_ptr(), c.stream()));
    return THPVariable_Wrap(dx);
  });
}

// y, pair_pos, weights, out
PyObject* unsort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled() && (needs_gradient(a[0]) || needs_gradient(a[2])))
      return in_graph("unsort_tokens", a, n);
    Call c;
    const at::Tensor& y = tensor(a[0], "y");
    const at::Tensor& pos = tensor(a[1], "pair_pos");
    const int64_t k = c.slots(pos, "pair_pos"), M = pos.size(0);
    c.dense(pos, at::kInt, "pair_pos", {M, k});
    const at::Tensor& w = tensor(a[2], "topk_weights");
    c.dense(w, at::kFloat, "topk_weights", {M, k});
    const long long ld = c.rows(y, "y");
    const int64_t H = y.size(1);
    if (y.size(0) != M * k) fail_shape("y", {M * k, H}, y.sizes());
    const at::Tensor out = c.out(a[3], y.scalar_type(), "out", {M, H});
    check_rc("moe_unsort_tokens",
             moe_unsort_tokens(y.data_ptr(), dtype_code(y.scalar_type()), ld, i32(pos), f32(w),
                               small(M), small(H), small(k), out.data_ptr(), c.stream()));
    return THPVariable_Wrap(out);
  });
}

// dout, y, sorted_pair, pair_pos, weights, dy, dweights
PyObject* unsort_tokens_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const at::Tensor& dout = tensor(a[0], "dout");
    const at::Tensor& y = tensor(a[1], "y");
    const at::Tensor& pair = tensor(a[2], "sorted_pair");
    const at::Tensor& pos = tensor(a[3], "pair_pos");
    const at::Tensor& w = tensor(a[4], "topk_weights");
    const int64_t k = c.slots(pos, "pair_pos"), M = pos.size(0);
    c.dense(pos, at::kInt, "pair_pos", {M, k});
    c.dense(pair, at::kInt, "sorted_pair", {M * k});
    c.dense(w, at::kFloat, "topk_weights", {M, k});
    const long long ldy = c.rows(y, "y");
    const int64_t H = y.size(1);
    if (y.size(0) != M * k) fail_shape("y", {M * k, H}, y.sizes());
    const long long ldd = c.rows(dout, "dout", M, H);
    if (dout.scalar_type() != y.scalar_type()) fail("dout, y: need one dtype");
    const at::Tensor dy = c.out(a[5], y.scalar_type(), "dy", {M * k, H});
    const at::Tensor dw = c.out(a[6], at::kFloat, "dweights", {M, k});
    check_rc("moe_unsort_tokens_backward",
             moe_unsort_tokens_backward(dout.data_ptr(), ldd, y.data_ptr(), ldy,
                                        dtype_code(y.scalar_type()), i32(pair), i32(pos), f32(w),
                                        small(M), small(H), small(k), dy.data_ptr(), f32(dw),
                                        c.stream()));
    return pack({dy, dw});
  });
}

// x, w, lora_a, lora_b, ids, scales, base, out, workspace
PyObject* lora_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled())
      for (int i : {0, 1, 2, 3, 5, 6})  // x, w, lora_a, lora_b, scales, base
        if (needs_gradient(a[i])) return in_graph("lora_linear", a, n);
    Call c;
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& A = tensor(a[2], "lora_a");
    const at::Tensor& B = tensor(a[3], "lora_b");
    const at::Tensor& ids = tensor(a[4], "adapter_ids");
    const at::Tensor& scales = tensor(a[5], "scales");
    const long long ldx = c.rows(x, "x");
    const at::ScalarType type = x.scalar_type();
    if (A.dim() != 3 || B.dim() != 3) fail("lora_a, lora_b: need [L][R][K] and [L][N][R]");
    const int64_t M = x.size(0), K = x.size(1), L = A.size(0), R = A.size(1), N = B.size(1);
    c.dense(A, type, "lora_a", {L, R, K});
    c.dense(B, type, "lora_b", {L, N, R});
    c.dense(ids, at::kInt, "adapter_ids", {M});
    c.dense(scales, at::kFloat, "scales", {L});
    const void *w = nullptr, *base = nullptr;
    long long ldb = 0;
    if (a[1] != Py_None) {
      const at::Tensor& t = tensor(a[1], "w");
      c.dense(t, type, "w", {N, K});
      w = t.data_ptr();
    }
    if (a[6] != Py_None) {
      const at::Tensor& t = tensor(a[6], "base");
      ldb = c.rows(t, "base", M, N);
      if (t.scalar_type() != type) fail("x, base: need one dtype");
      base = t.data_ptr();
    }
    const at::Tensor out = c.out(a[7], type, "out", {M, N});
    const at::Tensor ws = c.space(
        a[8], qmoe_lora_workspace_size(small(M), small(K), small(N), small(R), small(L)), kLora);
    check_rc("qmoe_lora_linear",
             qmoe_lora_linear(x.data_ptr(), dtype_code(type), ldx, w, A.data_ptr(), B.data_ptr(),
                              i32(ids), f32(scales), base, ldb, out.data_ptr(), small(M), small(K),
                              small(N), small(R), small(L), ws.data_ptr(), (size_t)ws.numel(),
                              c.stream()));
    if (a[8] == Py_None && M > 0) c.kept(kLora) = ws;
    return THPVariable_Wrap(out);
  });
}

// The kept workspaces of the current device.
PyObject* default_workspaces(PyObject*, PyObject* const*, Py_ssize_t n) {
  return guarded(n, 0, [&]() -> PyObject* {
    Call c;
    c.dev = c10::cuda::current_device();
    PyObject* r = PyList_New(0);
    if (!r) throw Raised{};
    for (int which = 0; which < kKeptKinds; ++which) {
      const at::Tensor& t = c.kept((Kept)which);
      if (!t.defined()) continue;
      PyObject* o = THPVariable_Wrap(t);
      const int rc = o ? PyList_Append(r, o) : -1;
      Py_XDECREF(o);
      if (rc != 0) {
        Py_DECREF(r);
        throw Raised{};
      }
    }
    return r;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XINCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

PyObject* set_graph(PyObject*, PyObject* f) {
  Py_XINCREF(f);
  Py_XSETREF(g_graph, f);
  Py_RETURN_NONE;
}

#define FAST(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {FAST(gate),
                          FAST(gate_backward),
                          FAST(sort_tokens),
                          FAST(sort_tokens_backward),
                          FAST(unsort_tokens),
                          FAST(unsort_tokens_backward),
                          FAST(lora_linear),
                          FAST(default_workspaces),
                          {"set_error", set_error, METH_O, nullptr},
                          {"set_graph", set_graph, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "qmoe_torch", nullptr, -1, kMethods,
                       nullptr,              nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qmoe_torch(void) { return PyModule_Create(&kModule); }
