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
#include <c10/core/AutogradState.h>
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
enum Kept { kSort, kLora, kFfn, kFfnBackward, kKeptKinds };
constexpr int kDevices = 64;

// The device of a call: every tensor has to be on the current one.
struct Call {
  static constexpr int kMostOutputs = 4;
  c10::DeviceIndex dev = -1;
  c10::TensorImpl* into[kMostOutputs];  // given outputs
  int written = 0;
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
    // its history would stand for values that are no longer there
    if (c10::GradMode::is_enabled() && t.requires_grad())
      fail(std::string(name) + ": an output to write into cannot require a gradient (or call it "
                               "under torch.no_grad())");
    if (written == kMostOutputs) fail("too many outputs");
    into[written++] = t.unsafeGetTensorImpl();
    return t;
  }
  // The library's answer to the call; where it was taken, autograd is told of the outputs that were
  // written into, so that a node that has kept one of them does not take it for what it was.
  void answer(const char* fn, int rc) {
    check_rc(fn, rc);
    for (int i = 0; i < written; ++i)
      if (!into[i]->is_inference()) into[i]->bump_version();
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
  // What has the error word of the last call that brought no workspace (one per operator
  // and device; never destroyed, since that could come after the CUDA context's end).
  at::Tensor& kept(Kept which) const {
    static auto* all = new std::array<at::Tensor, kDevices * kKeptKinds>();
    if (dev < 0 || dev >= kDevices) fail("too many CUDA devices");
    return (*all)[(size_t)(dev * kKeptKinds + which)];
  }
  // Where a call without a workspace has its error word, kept until the next such call: the start
  // of its workspace, but of one past 1 MiB, which is not to be held for that, a word of its own.
  static constexpr int64_t kMostHeld = 1 << 20;
  at::Tensor error_word(const at::Tensor& ws) {
    return ws.numel() <= kMostHeld ? ws : make(at::kByte, {256});
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

// No call has a derivative in forward mode: a tangent is refused, not dropped.  (Tensors that autograd
// has had nothing to do with are passed over by a look at a pointer.)
bool carries_tangent(PyObject* const* a, Py_ssize_t n) {
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* const o = a[i];
    if (o == Py_None || PyBool_Check(o) || PyLong_CheckExact(o) || PyFloat_CheckExact(o) ||
        !THPVariable_Check(o))
      continue;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.unsafeGetTensorImpl()->autograd_meta() && t._fw_grad(0).defined())
      return c10::AutogradState::get_tls_state().get_fw_grad_mode();
  }
  return false;
}

template <class F>
PyObject* guarded(PyObject* const* a, Py_ssize_t given, Py_ssize_t wanted, F&& body) {
  HANDLE_TH_ERRORS
  if (given != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (carries_tangent(a, given)) {
    PyErr_SetString(PyExc_NotImplementedError,
                    "no derivative in forward mode: call it on tensors without a tangent");
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
  return guarded(a, n, 10, [&]() -> PyObject* {
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
    c.answer("moe_gate",
             moe_gate(logits.data_ptr(), dtype_code(logits.scalar_type()), ld, small(M), small(E),
                      (int)k, small(integer(a[2])), bias, small(integer(a[4])),
                      small(integer(a[5])), truth(a[6]), (float)scale, i32_out(ids),
                      f32(w), c.stream()));
    return pack({ids, w});
  });
}

// dweights, logits, ids, scoring, renormalize, scale, dlogits
PyObject* gate_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 7, [&]() -> PyObject* {
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
    c.answer("moe_gate_backward",
             moe_gate_backward(f32(dw), logits.data_ptr(), dtype_code(logits.scalar_type()), ld,
                               i32(ids), small(M), small(E), small(k), small(integer(a[3])),
                               truth(a[4]), (float)scale, dl.data_ptr(), c.stream()));
    return THPVariable_Wrap(dl);
  });
}

// x, ids, E, xs, workspace
PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 5, [&]() -> PyObject* {
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
    c.answer("moe_sort_tokens",
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
  return guarded(a, n, 3, [&]() -> PyObject* {
    Call c;
    const at::Tensor& y = tensor(a[0], "dxs");
    const at::Tensor& pos = tensor(a[1], "pair_pos");
    const int64_t k = c.slots(pos, "pair_pos"), M = pos.size(0);
    c.dense(pos, at::kInt, "pair_pos", {M, k});
    const long long ld = c.rows(y, "dxs");
    const int64_t H = y.size(1);
    if (y.size(0) != M * k) fail_shape("dxs", {M * k, H}, y.sizes());
    const at::Tensor dx = c.out(a[2], y.scalar_type(), "dx", {M, H});
    c.answer("moe_sort_tokens_backward",
             moe_sort_tokens_backward(y.data_ptr(), dtype_code(y.scalar_type()), ld, i32(pos),
                                      small(M), small(H), small(k), dx.data_ptr(), c.stream()));
    return THPVariable_Wrap(dx);
  });
}

// y, pair_pos, weights, out
PyObject* unsort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 4, [&]() -> PyObject* {
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
    c.answer("moe_unsort_tokens",
             moe_unsort_tokens(y.data_ptr(), dtype_code(y.scalar_type()), ld, i32(pos), f32(w),
                               small(M), small(H), small(k), out.data_ptr(), c.stream()));
    return THPVariable_Wrap(out);
  });
}

// dout, y, sorted_pair, pair_pos, weights, dy, dweights
PyObject* unsort_tokens_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 7, [&]() -> PyObject* {
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
    c.answer("moe_unsort_tokens_backward",
             moe_unsort_tokens_backward(dout.data_ptr(), ldd, y.data_ptr(), ldy,
                                        dtype_code(y.scalar_type()), i32(pair), i32(pos), f32(w),
                                        small(M), small(H), small(k), dy.data_ptr(), f32(dw),
                                        c.stream()));
    return pack({dy, dw});
  });
}

// x, w, lora_a, lora_b, ids, scales, base, out, workspace
PyObject* lora_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 9, [&]() -> PyObject* {
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
    c.answer("qmoe_lora_linear",
             qmoe_lora_linear(x.data_ptr(), dtype_code(type), ldx, w, A.data_ptr(), B.data_ptr(),
                              i32(ids), f32(scales), base, ldb, out.data_ptr(), small(M), small(K),
                              small(N), small(R), small(L), ws.data_ptr(), (size_t)ws.numel(),
                              c.stream()));
    if (a[8] == Py_None && M > 0) c.kept(kLora) = ws;
    return THPVariable_Wrap(out);
  });
}

bool given(PyObject* o) { return o != Py_None; }
void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw Raised{};
  return v;
}
PyObject* wrap_or_none(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
PyObject* pack_some(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap_or_none(t));
  return r;
}

// What the forward and backward calls of the norms around a block have in common.
struct Norms {
  int type = 0, weight_type = 0;
  int64_t M = 0, H = 0;
  at::Tensor gate, post, pre;
  int gate_type = 0, gate_form = 0, gating = 0;
  long long ldgate = 0;

  // gate, gating, post_weight, pre_weight
  void take(Call& c, const at::Tensor& y, PyObject* g, PyObject* how, PyObject* post_weight,
            PyObject* pre_weight) {
    M = y.size(0), H = y.size(1);
    type = gate_type = weight_type = dtype_code(y.scalar_type());
    gating = small(integer(how));
    if (given(g)) {
      gate = tensor(g, "gate");
      gate_type = of_either(y, gate, "gate");
      if (gate.dim() != 2 || gate.layout() != at::kStrided)
        fail("gate: need [M][1], [1][H] or [M][H]");
      const int64_t n = gate.size(0), w = gate.size(1);
      if (n == M && w == 1) {  // (also of a row of one element)
        gate_form = QMOE_GATE_TOKEN;
        c.here(gate, "gate");
        ldgate = M > 1 ? gate.stride(0) : 1;
      } else if (n == 1 && w == H) {
        gate_form = QMOE_GATE_CHANNEL;
        c.rows(gate, "gate");
      } else {
        gate_form = QMOE_GATE_FULL;
        ldgate = c.rows(gate, "gate", M, H);
      }
    }
    vector(c, y, post_weight, "post_weight", &post);
    vector(c, y, pre_weight, "pre_weight", &pre);
    if (post.defined() && pre.defined() && post.scalar_type() != pre.scalar_type())
      fail("post_weight, pre_weight: need one dtype");
  }
  static int of_either(const at::Tensor& y, const at::Tensor& t, const char* name) {
    if (t.scalar_type() != y.scalar_type() && t.scalar_type() != at::kFloat)
      fail(std::string(name) + ": need the activations' dtype or fp32");
    return dtype_code(t.scalar_type());
  }
  void vector(Call& c, const at::Tensor& y, PyObject* o, const char* name, at::Tensor* to) {
    if (!given(o)) return;
    *to = tensor(o, name);
    weight_type = of_either(y, *to, name);
    c.dense(*to, to->scalar_type(), name, {H});
  }
};

// y, residual, gate, gating, post_weight, pre_weight, residual_scale, weight_offset, eps, out,
// normed
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 11, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled())
      for (int i : {0, 1, 2, 4, 5})
        if (needs_gradient(a[i])) return in_graph("block_norm", a, n);
    Call c;
    const at::Tensor& y = tensor(a[0], "y");
    const long long ldy = c.rows(y, "y");
    const at::ScalarType type = y.scalar_type();
    Norms s;
    s.take(c, y, a[2], a[3], a[4], a[5]);
    at::Tensor residual, out, normed, post_rstd, pre_rstd;
    long long ldr = 0;
    if (given(a[1])) {
      residual = tensor(a[1], "residual");
      ldr = c.rows(residual, "residual", s.M, s.H);
      if (residual.scalar_type() != type) fail("y, residual: need one dtype");
    }
    const bool changes = residual.defined() || s.gate.defined() || s.post.defined();
    if (!changes && !s.pre.defined()) fail("block_norm: nothing to compute");
    if (!changes && given(a[9])) fail("out: would be y");
    if (!s.pre.defined() && given(a[10])) fail("normed: needs pre_weight");
    if (changes) out = c.out(a[9], type, "out", {s.M, s.H});
    if (s.pre.defined()) {
      normed = c.out(a[10], type, "normed", {s.M, s.H});
      pre_rstd = c.make(at::kFloat, {s.M});
    }
    if (s.post.defined()) post_rstd = c.make(at::kFloat, {s.M});
    c.answer("qmoe_block_norm",
             qmoe_block_norm(y.data_ptr(), s.type, ldy, data(residual), ldr, (float)real(a[6]),
                             data(s.gate), s.gate_type, s.gate_form, s.ldgate, s.gating,
                             data(s.post), data(s.pre), s.weight_type, (float)real(a[7]),
                             (float)real(a[8]), small(s.M), small(s.H), data(out), data(normed),
                             static_cast<float*>(data(post_rstd)),
                             static_cast<float*>(data(pre_rstd)), c.stream()));
    return pack_some({out, normed, post_rstd, pre_rstd});
  });
}

// dout, dnormed, y, out, gate, gating, post_weight, pre_weight, residual_scale, weight_offset,
// post_rstd, pre_rstd, which of the gradients are wanted: residual, gate, post_weight, pre_weight;
// whether a full gate's is of the gate's type (else of y's)
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 17, [&]() -> PyObject* {
    Call c;
    const at::Tensor& y = tensor(a[2], "y");
    const long long ldy = c.rows(y, "y");
    const at::ScalarType type = y.scalar_type();
    Norms s;
    s.take(c, y, a[4], a[5], a[6], a[7]);
    at::Tensor dout, dnormed, out, rstd[2], dresidual, dgate, dpost, dpre;
    long long ldd = 0, ldn = 0, ldo = 0;
    auto rows = [&](PyObject* o, const char* name, at::Tensor* t, long long* ld) {
      if (!given(o)) return;
      *t = tensor(o, name);
      *ld = c.rows(*t, name, s.M, s.H);
      if (t->scalar_type() != type) fail(std::string(name) + ": need y's dtype");
    };
    rows(a[0], "dout", &dout, &ldd);
    rows(a[1], "dnormed", &dnormed, &ldn);
    rows(a[3], "out", &out, &ldo);
    const char* names[2] = {"post_rstd", "pre_rstd"};
    for (int i = 0; i < 2; ++i) {
      if (!given(a[10 + i])) continue;
      rstd[i] = tensor(a[10 + i], names[i]);
      c.dense(rstd[i], at::kFloat, names[i], {s.M});
    }
    if (!dout.defined() && !dnormed.defined()) fail("dout, dnormed: need one of them");
    if (s.pre.defined() != dnormed.defined()) fail("dnormed: goes with pre_weight");
    const at::Tensor dy = c.make(type, {s.M, s.H});
    if (truth(a[12])) dresidual = c.make(type, {s.M, s.H});
    const bool own = s.gate_form == QMOE_GATE_FULL && truth(a[16]);
    if (truth(a[13]) && s.gate.defined())
      dgate = s.gate_form == QMOE_GATE_FULL ? c.make(own ? s.gate.scalar_type() : type, {s.M, s.H})
              : s.gate_form == QMOE_GATE_TOKEN ? c.make(at::kFloat, {s.M, 1})
                                               : c.make(at::kFloat, {1, s.H});
    if (truth(a[14]) && s.post.defined()) dpost = c.make(at::kFloat, {s.H});
    if (truth(a[15]) && s.pre.defined()) dpre = c.make(at::kFloat, {s.H});
    const size_t bytes = qmoe_block_norm_backward_workspace_size(small(s.M), small(s.H));
    const at::Tensor ws = c.make(at::kByte, {(int64_t)(bytes < 256 ? 256 : bytes)});
    c.answer("qmoe_block_norm_backward",
             qmoe_block_norm_backward(
                 data(dout), ldd, data(dnormed), ldn, y.data_ptr(), s.type, ldy, data(out), ldo,
                 (float)real(a[8]), data(s.gate), s.gate_type,
                 s.gate_form + (own ? QMOE_GATE_OWN_GRADIENT : 0), s.ldgate, s.gating, data(s.post),
                 data(s.pre), s.weight_type, (float)real(a[9]), static_cast<float*>(data(rstd[0])),
                 static_cast<float*>(data(rstd[1])), small(s.M), small(s.H), dy.data_ptr(),
                 data(dresidual), data(dgate),
                 static_cast<float*>(data(dpost)), static_cast<float*>(data(dpre)), ws.data_ptr(),
                 (size_t)ws.numel(), c.stream()));
    return pack_some({dy, dresidual, dgate, dpost, dpre});
  });
}

// x, codes, scales
PyObject* checkpoint8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 3, [&]() -> PyObject* {
    Call c;
    const at::Tensor& x = tensor(a[0], "x");
    const long long ldx = c.rows(x, "x");
    const int64_t M = x.size(0), C = x.size(1);
    const at::Tensor codes = c.out(a[1], at::kChar, "codes", {M, C});
    const at::Tensor scales = c.out(a[2], at::kByte, "scales", {M, (C + 31) / 32});
    c.answer("qmoe_checkpoint8",
             qmoe_checkpoint8(x.data_ptr(), dtype_code(x.scalar_type()), ldx, small(M), small(C),
                              static_cast<int8_t*>(codes.data_ptr()),
                              static_cast<uint8_t*>(scales.data_ptr()), c.stream()));
    return pack({codes, scales});
  });
}

// A checkpoint's codes and scales, `parts` matrices beside each other.
const int8_t* codes_of(Call& c, const at::Tensor& codes, const at::Tensor& scales, int64_t M,
                       int64_t C, int parts, const char* name) {
  c.dense(codes, at::kChar, (std::string(name) + " codes").c_str(), {M, parts * C});
  c.dense(scales, at::kByte, (std::string(name) + " scales").c_str(), {M, parts * ((C + 31) / 32)});
  return static_cast<const int8_t*>(codes.data_ptr());
}

// codes, scales, an empty tensor of the wanted type, out
PyObject* checkpoint8_restore(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 4, [&]() -> PyObject* {
    Call c;
    const at::Tensor& codes = tensor(a[0], "codes");
    const at::Tensor& scales = tensor(a[1], "scales");
    if (codes.dim() != 2) fail("codes: need [M][C]");
    const int64_t M = codes.size(0), C = codes.size(1);
    const int8_t* p = codes_of(c, codes, scales, M, C, 1, "x");
    const at::ScalarType type = tensor(a[2], "dtype").scalar_type();
    if (dtype_code(type) < 0) fail("dtype: need bf16, fp16 or fp32");
    const at::Tensor out = c.out(a[3], type, "out", {M, C});
    c.answer("qmoe_checkpoint8_restore",
             qmoe_checkpoint8_restore(p, static_cast<const uint8_t*>(scales.data_ptr()),
                                      dtype_code(type), small(M), small(C), out.data_ptr(),
                                      c.stream()));
    return THPVariable_Wrap(out);
  });
}

// The sizes of a gated feed-forward block by its weights.
struct Ffn {
  at::ScalarType type;
  int64_t H, I;
  Ffn(Call& c, const at::Tensor& w13, const at::Tensor& w2) {
    if (w13.dim() != 2 || w2.dim() != 2) fail("w13, w2: need [2I][H] and [H][I]");
    type = w2.scalar_type();
    H = w2.size(0), I = w2.size(1);
    if (type != at::kBFloat16 && type != at::kHalf) fail("w13, w2: need bf16 or fp16");
    c.dense(w13, type, "w13", {2 * I, H});
    c.dense(w2, type, "w2", {H, I});
  }
  long long rows(Call& c, const at::Tensor& t, const char* name, int64_t M) const {
    const long long ld = c.rows(t, name, M, H);
    if (t.scalar_type() != type) fail(std::string(name) + ": need the weights' dtype");
    return ld;
  }
};

// x, w13, w2, activation, limit, what is kept (0: nothing, 16, 8), out, workspace, what a node of
// autograd's graph keeps (16, 8; 0: its backward pass is its caller's)
PyObject* gated_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 9, [&]() -> PyObject* {
    if (c10::GradMode::is_enabled())
      for (int i : {0, 1, 2})  // x, w13, w2
        if (needs_gradient(a[i]))
          return in_graph(integer(a[8]) != 0 ? "gated_ffn" : "gated_ffn_saved", a, n);
    Call c;
    const at::Tensor& x = tensor(a[0], "x");
    const at::Tensor& w13 = tensor(a[1], "w13");
    const at::Tensor& w2 = tensor(a[2], "w2");
    const Ffn f(c, w13, w2);
    if (x.dim() != 2) fail("x: need [M][H]");
    const int64_t M = x.size(0);
    const long long ldx = f.rows(c, x, "x", M);
    const int64_t keep = integer(a[5]);
    at::Tensor kept, scales;
    if (keep == 16) kept = c.make(f.type, {M, 2 * f.I});
    if (keep == 8) {
      kept = c.make(at::kChar, {M, 2 * f.I});
      scales = c.make(at::kByte, {M, 2 * ((f.I + 31) / 32)});
    }
    const at::Tensor out = c.out(a[6], f.type, "out", {M, f.H});
    const at::Tensor ws =
        c.space(a[7], qmoe_gated_ffn_workspace_size(small(M), small(f.H), small(f.I)), kFfn);
    const at::Tensor error = given(a[7]) ? ws : c.error_word(ws);
    c.answer("qmoe_gated_ffn",
             qmoe_gated_ffn_error_at(
                 x.data_ptr(), dtype_code(f.type), ldx, w13.data_ptr(), w2.data_ptr(),
                 small(integer(a[3])), (float)real(a[4]), small(M), small(f.H), small(f.I),
                 out.data_ptr(), data(kept), static_cast<uint8_t*>(data(scales)), ws.data_ptr(),
                 (size_t)ws.numel(), static_cast<uint32_t*>(error.data_ptr()), c.stream()));
    if (!given(a[7]) && M > 0) c.kept(kFfn) = error;
    if (keep == 0) return THPVariable_Wrap(out);
    return pack_some({out, kept, scales});
  });
}

// dout, x or its codes, x's scales or None, w13, w2, kept, kept's scales or None, activation, limit,
// which of the gradients are wanted: x, w13, w2; workspace
PyObject* gated_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 13, [&]() -> PyObject* {
    Call c;
    const at::Tensor& dout = tensor(a[0], "dout");
    const at::Tensor& x = tensor(a[1], "x");
    const at::Tensor& w13 = tensor(a[3], "w13");
    const at::Tensor& w2 = tensor(a[4], "w2");
    const at::Tensor& kept = tensor(a[5], "kept");
    const Ffn f(c, w13, w2);
    if (dout.dim() != 2) fail("dout: need [M][H]");
    const int64_t M = dout.size(0);
    const long long ldd = f.rows(c, dout, "dout", M);
    long long ldx = f.H;
    at::Tensor xs, ks;
    if (given(a[2]) != given(a[6])) fail("x, kept: both in 8 bits, or neither");
    if (given(a[2])) {
      xs = tensor(a[2], "x scales");
      ks = tensor(a[6], "kept scales");
      codes_of(c, x, xs, M, f.H, 1, "x");
      codes_of(c, kept, ks, M, f.I, 2, "kept");
    } else {
      ldx = f.rows(c, x, "x", M);
      c.dense(kept, f.type, "kept", {M, 2 * f.I});
    }
    at::Tensor dx, dw13, dw2;
    if (truth(a[9])) dx = c.make(f.type, {M, f.H});
    if (truth(a[10])) dw13 = c.make(f.type, {2 * f.I, f.H});
    if (truth(a[11])) dw2 = c.make(f.type, {f.H, f.I});
    const at::Tensor ws = c.space(
        a[12], qmoe_gated_ffn_backward_workspace_size(small(M), small(f.H), small(f.I),
                                                      xs.defined() ? 8 : 16), kFfnBackward);
    const at::Tensor error = given(a[12]) ? ws : c.error_word(ws);
    c.answer("qmoe_gated_ffn_backward",
             qmoe_gated_ffn_backward_error_at(
                 dout.data_ptr(), dtype_code(f.type), ldd, x.data_ptr(), ldx,
                 static_cast<uint8_t*>(data(xs)), w13.data_ptr(), w2.data_ptr(), kept.data_ptr(),
                 static_cast<uint8_t*>(data(ks)), small(integer(a[7])), (float)real(a[8]), small(M),
                 small(f.H), small(f.I), data(dx), data(dw13), data(dw2), ws.data_ptr(),
                 (size_t)ws.numel(), static_cast<uint32_t*>(error.data_ptr()), c.stream()));
    if (!given(a[12]) && M > 0) c.kept(kFfnBackward) = error;
    return pack_some({dx, dw13, dw2});
  });
}

// The kept workspaces of the current device.
PyObject* default_workspaces(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(a, n, 0, [&]() -> PyObject* {
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
                          FAST(block_norm),
                          FAST(block_norm_backward),
                          FAST(checkpoint8),
                          FAST(checkpoint8_restore),
                          FAST(gated_ffn),
                          FAST(gated_ffn_backward),
                          FAST(default_workspaces),
                          {"set_error", set_error, METH_O, nullptr},
                          {"set_graph", set_graph, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "qmoe_torch", nullptr, -1, kMethods,
                       nullptr,              nullptr,      nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_qmoe_torch(void) { return PyModule_Create(&kModule); }
