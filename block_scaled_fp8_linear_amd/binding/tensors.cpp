// The package's functions over include/fp8bl_int8.h and include/fp8bl_qkv.h:
// tensors checked, outputs and workspaces allocated, and the C call made on the
// current stream. No arithmetic.
//
// In C++ for the smallest calls, which take longer on the host than on the GPU:
// with the same checks in Python over ctypes, storing 16 tokens took 12.7 us of
// host time, 3.9 of them the launch.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/util/Exception.h>

#include <new>
#include <string>

#include "fp8bl_int8.h"
#include "fp8bl_qkv.h"

namespace {

using at::ScalarType;
using at::Tensor;

// ---- Errors: a Python exception on its way out of a call.
struct Raise {
  PyObject* type;        // null: the exception is set already
  std::string what;
};

[[noreturn]] void type_error(const std::string& what) { throw Raise{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Raise{PyExc_ValueError, what}; }

PyObject* g_error;        // the package's Fp8blError
PyObject* g_raw_stream;   // torch's current stream of a device, as a number
PyObject* g_memory;       // torch's OutOfMemoryError

// Makes a call, other threads running meanwhile: a launch can wait for the GPU.
template <typename F>
void run(const char* where, F call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  if (status == FP8BL_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raise{nullptr, {}};
}

hipStream_t stream_of(int64_t idx) {
  PyObject* n = PyLong_FromLongLong(idx);
  PyObject* s = n ? PyObject_CallOneArg(g_raw_stream, n) : nullptr;
  Py_XDECREF(n);
  void* p = s ? PyLong_AsVoidPtr(s) : nullptr;
  Py_XDECREF(s);
  if (p == nullptr && PyErr_Occurred()) throw Raise{nullptr, {}};
  return static_cast<hipStream_t>(p);
}

// A new tensor beside `like`, from torch's allocator without its dispatcher (0.25 us
// less each: the backward pass of 77 tokens 11.0 -> 9.8 us of host time).
Tensor fresh(at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}

std::string dtype_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Char: return "torch.int8";
    case ScalarType::Byte: return "torch.uint8";
    default: return std::string("torch ") + c10::toString(t);
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

// ---- Parameters by position and by name.
constexpr int kMaxParams = 20;

struct Signature {
  const char* name;
  int required, count;
  const char* params[kMaxParams];
  const char* backward = nullptr;     // its backward function, where there is one
  PyObject* interned[kMaxParams] = {};
};

struct Args {
  const Signature& s;
  PyObject* v[kMaxParams] = {};

  Args(const Signature& sig, PyObject* const* args, Py_ssize_t n, PyObject* names) : s(sig) {
    if (n > s.count) type_error(std::string(s.name) + "() takes at most " + std::to_string(s.count) + " arguments");
    for (Py_ssize_t i = 0; i < n; ++i) v[i] = args[i];
    const Py_ssize_t k = names ? PyTuple_GET_SIZE(names) : 0;
    for (Py_ssize_t i = 0; i < k; ++i) {
      PyObject* name = PyTuple_GET_ITEM(names, i);
      int at = -1;
      for (int j = 0; j < s.count && at < 0; ++j)
        if (s.interned[j] == name) at = j;
      for (int j = 0; j < s.count && at < 0; ++j)
        if (PyUnicode_Compare(s.interned[j], name) == 0) at = j;
      const char* text = PyUnicode_AsUTF8(name);
      if (at < 0) type_error(std::string(s.name) + "() got an unexpected keyword argument '" + (text ? text : "") + "'");
      if (v[at]) type_error(std::string(s.name) + "() got multiple values for argument '" + s.params[at] + "'");
      v[at] = args[n + i];
    }
    for (int i = 0; i < s.required; ++i)
      if (!v[i]) type_error(std::string(s.name) + "() missing argument '" + s.params[i] + "'");
  }
  bool given(int i) const { return v[i] != nullptr && v[i] != Py_None; }
  const Tensor& tensor(int i) const {
    if (!v[i] || !THPVariable_Check(v[i])) type_error(std::string(s.params[i]) + " must be a tensor");
    return THPVariable_Unpack(v[i]);
  }
  bool truth(int i, bool otherwise) const {
    if (!v[i]) return otherwise;
    const int t = PyObject_IsTrue(v[i]);
    if (t < 0) throw Raise{nullptr, {}};
    return t != 0;
  }
  double number(int i, double otherwise) const {
    if (!v[i]) return otherwise;
    const double d = PyFloat_AsDouble(v[i]);
    if (d == -1.0 && PyErr_Occurred()) throw Raise{nullptr, {}};
    return d;
  }
  // Nothing here is recorded by autograd: a tensor that asks for a gradient, be it
  // read or written, would lose it without a word, so it is refused.
  // A tangent (forward mode, which no_grad leaves on) is refused likewise.
  void outside_autograd() const {
    const bool grad = c10::GradMode::is_enabled();
    for (int i = 0; i < s.count; ++i) {
      if (!v[i] || !THPVariable_Check(v[i])) continue;
      const Tensor& t = THPVariable_Unpack(v[i]);
      if (t.unsafeGetTensorImpl()->autograd_meta() == nullptr) continue;     // neither
      if (t._fw_grad(0).defined())
        throw Raise{PyExc_RuntimeError,
                    std::string(s.name) + " is not recorded by autograd and " + s.params[i] + " has a tangent: unpack it first"};
      if (grad && t.requires_grad())
        throw Raise{PyExc_RuntimeError,
                    std::string(s.name) + " is not recorded by autograd and " + s.params[i] + " requires grad: call it " +
                        (s.backward ? std::string("in a torch.autograd.Function with ") + s.backward + ", or " : "") +
                        "under torch.no_grad()" + (s.backward ? "" : " (there is no backward function)")};
    }
  }
  int64_t device(int i) const {
    const Tensor& t = tensor(i);
    if (!t.is_cuda()) type_error(std::string(s.params[i]) + " must be a device tensor");
    return t.get_device();
  }
  // The address of a contiguous array of the call's device.
  void* array(int i, ScalarType dtype, at::IntArrayRef shape, int64_t idx) const {
    const Tensor& t = tensor(i);
    const std::string name = s.params[i];
    if (t.scalar_type() != dtype) type_error(name + " must be " + dtype_name(dtype) + ", got " + dtype_name(t.scalar_type()));
    if (!t.is_cuda()) type_error(name + " must be a device tensor");
    if (t.sizes() != shape) value_error(name + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (!t.is_contiguous()) value_error(name + " must be contiguous");
    if (t.get_device() != idx) value_error(name + " is on " + t.device().str() + ", expected cuda:" + std::to_string(idx));
    return t.data_ptr();
  }
  void* optional(int i, ScalarType dtype, at::IntArrayRef shape, int64_t idx) const {
    return given(i) ? array(i, dtype, shape, idx) : nullptr;
  }
  // bf16 [tokens, heads, head_dim] with its strides.
  fp8bl_heads heads(int i, at::IntArrayRef shape, int64_t idx) const {
    const Tensor& t = tensor(i);
    const std::string name = s.params[i];
    if (t.scalar_type() != ScalarType::BFloat16) type_error(name + " must be torch.bfloat16, got " + dtype_name(t.scalar_type()));
    if (!t.is_cuda()) type_error(name + " must be a device tensor");
    if (t.sizes() != shape) value_error(name + " must be " + shape_text(shape) + ", got " + shape_text(t.sizes()));
    if (t.get_device() != idx) value_error(name + " is on " + t.device().str() + ", expected cuda:" + std::to_string(idx));
    if (t.stride(2) != 1) value_error(name + " must have its last axis contiguous");
    return fp8bl_heads{static_cast<uint16_t*>(t.data_ptr()), t.stride(0), t.stride(1)};
  }
  at::IntArrayRef matrix(int i) const {
    const Tensor& t = tensor(i);
    if (t.dim() != 2) value_error(std::string(s.params[i]) + " must be a matrix, got " + shape_text(t.sizes()));
    return t.sizes();
  }
  at::IntArrayRef head_shape(int i) const {
    const Tensor& t = tensor(i);
    if (t.dim() != 3)
      value_error(std::string(s.params[i]) + " must be [tokens, heads, head_dim], got " + shape_text(t.sizes()));
    return t.sizes();
  }
};

// A caller's tensor was written: autograd tells by its version that what it saved is
// no longer there. (Inference tensors have none.)
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// An output: the one given, or a new tensor.
struct Output {
  PyObject* object = nullptr;
  bool given = false;
  Output(const Args& a, int i, at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
    if (a.given(i)) {
      a.tensor(i);
      object = a.v[i];
      given = true;
      Py_INCREF(object);
    } else {
      object = THPVariable_Wrap(fresh(shape, dtype, like));
      if (!object) throw Raise{nullptr, {}};
    }
  }
  Output(at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
    object = THPVariable_Wrap(fresh(shape, dtype, like));
    if (!object) throw Raise{nullptr, {}};
  }
  Output() = default;
  Output(const Output&) = delete;
  Output& operator=(const Output&) = delete;
  ~Output() { Py_XDECREF(object); }
  // The output for the caller, once the call that writes it is on its way.
  PyObject* release() {
    if (given) written(THPVariable_Unpack(object));
    PyObject* o = object;
    object = nullptr;
    if (!o) {
      o = Py_None;
      Py_INCREF(o);
    }
    return o;
  }
  const Tensor& tensor() const { return THPVariable_Unpack(object); }
};

// `a` with an output in the place of parameter i, for the checks.
struct With {
  Args& a;
  int i;
  PyObject* was;
  With(Args& args, int at, const Output& o) : a(args), i(at), was(args.v[at]) { a.v[at] = o.object; }
  ~With() { a.v[i] = was; }
};

struct Workspace {
  Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(const Args& a, int i, size_t need, int64_t idx, const Tensor& like) {
    if (a.given(i)) {
      const Tensor& t = a.tensor(i);
      if (!t.is_cuda() || t.get_device() != idx || !t.is_contiguous())
        value_error("workspace must be a contiguous tensor on cuda:" + std::to_string(idx));
      p = t.data_ptr();
      bytes = t.nbytes();
    } else if (need > 0) {
      own = fresh({(int64_t)need}, ScalarType::Byte, like);
      p = own.data_ptr();
      bytes = need;
    }
  }
};

PyObject* pair(Output& a, Output& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) throw Raise{nullptr, {}};
  PyTuple_SET_ITEM(t, 0, a.release());
  PyTuple_SET_ITEM(t, 1, b.release());
  return t;
}

// ---- 8-bit integer linear.

Signature kRowQuantize{"int8_row_quantize", 1, 3, {"x", "q", "scale"}};
PyObject* row_quantize(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& x = a.tensor(0);
  const c10::DeviceGuard guard(x.device());
  const bool bf16 = x.scalar_type() == ScalarType::BFloat16;
  if (!bf16 && x.scalar_type() != ScalarType::Float)
    type_error("x must be float32 or bfloat16, got " + dtype_name(x.scalar_type()));
  const int64_t m = a.matrix(0)[0], k = a.matrix(0)[1];
  Output q(a, 1, {m, k}, ScalarType::Char, x), scale(a, 2, {m}, ScalarType::Float, x);
  const With wq(a, 1, q), ws(a, 2, scale);
  void* const xp = a.array(0, x.scalar_type(), {m, k}, idx);
  int8_t* const qp = static_cast<int8_t*>(a.array(1, ScalarType::Char, {m, k}, idx));
  float* const sp = static_cast<float*>(a.array(2, ScalarType::Float, {m}, idx));
  const hipStream_t st = stream_of(idx);
  run("int8_row_quantize", [&] {
    return bf16 ? int8_row_quantize_bf16(static_cast<uint16_t*>(xp), qp, sp, m, k, st)
                : int8_row_quantize(static_cast<float*>(xp), qp, sp, m, k, st);
  });
  return pair(q, scale);
}

Signature kLinear{"int8_linear", 4, 7, {"xq", "x_scale", "wq", "w_scale", "bias", "out", "workspace"}};
PyObject* linear(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& x = a.tensor(0);
  const c10::DeviceGuard guard(x.device());
  const int64_t m = a.matrix(0)[0], k = a.matrix(0)[1], n = a.matrix(2)[0];
  Output out(a, 5, {m, n}, ScalarType::BFloat16, x);
  const With wo(a, 5, out);
  auto* xq = static_cast<int8_t*>(a.array(0, ScalarType::Char, {m, k}, idx));
  auto* xs = static_cast<float*>(a.array(1, ScalarType::Float, {m}, idx));
  auto* wq = static_cast<int8_t*>(a.array(2, ScalarType::Char, {n, k}, idx));
  auto* ws = static_cast<float*>(a.array(3, ScalarType::Float, {n}, idx));
  auto* bias = static_cast<uint16_t*>(a.optional(4, ScalarType::BFloat16, {n}, idx));
  auto* y = static_cast<uint16_t*>(a.array(5, ScalarType::BFloat16, {m, n}, idx));
  const Workspace w(a, 6, int8_linear_workspace_size(m, n, k), idx, x);
  const hipStream_t st = stream_of(idx);
  run("int8_linear", [&] { return int8_linear(xq, xs, wq, ws, bias, y, m, n, k, w.p, w.bytes, st); });
  return out.release();
}

Signature kLinearBf16{"int8_linear_bf16", 3, 6, {"x", "wq", "w_scale", "bias", "out", "workspace"}};
PyObject* linear_bf16(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& xt = a.tensor(0);
  const c10::DeviceGuard guard(xt.device());
  const int64_t m = a.matrix(0)[0], k = a.matrix(0)[1], n = a.matrix(1)[0];
  Output out(a, 4, {m, n}, ScalarType::BFloat16, xt);
  const With wo(a, 4, out);
  auto* x = static_cast<uint16_t*>(a.array(0, ScalarType::BFloat16, {m, k}, idx));
  auto* wq = static_cast<int8_t*>(a.array(1, ScalarType::Char, {n, k}, idx));
  auto* ws = static_cast<float*>(a.array(2, ScalarType::Float, {n}, idx));
  auto* bias = static_cast<uint16_t*>(a.optional(3, ScalarType::BFloat16, {n}, idx));
  auto* y = static_cast<uint16_t*>(a.array(4, ScalarType::BFloat16, {m, n}, idx));
  const Workspace w(a, 5, int8_linear_bf16_workspace_size(m, n, k), idx, xt);
  const hipStream_t st = stream_of(idx);
  run("int8_linear_bf16", [&] { return int8_linear_bf16(x, wq, ws, bias, y, m, n, k, w.p, w.bytes, st); });
  return out.release();
}

// ---- From the QKV projection to its cache.

// Norm and rotation: parameters `at` .. at + 3 are q_weight, k_weight, positions
// and inv_freq, and `how` .. how + 2 axes, eps and interleaved.
void set_turn(const Args& a, int at, int how, int64_t idx, fp8bl_qkv* g) {
  const int64_t d = g->head_dim, t = g->tokens;
  g->q_weight = static_cast<uint16_t*>(a.array(at, ScalarType::BFloat16, {d}, idx));
  g->k_weight = static_cast<uint16_t*>(a.array(at + 1, ScalarType::BFloat16, {d}, idx));
  const Tensor& pos = a.tensor(at + 2);
  if (pos.dim() == 1) {
    g->axes = 1;
    g->positions = static_cast<int32_t*>(a.array(at + 2, ScalarType::Int, {t}, idx));
  } else {
    g->axes = a.matrix(at + 2)[0];
    g->positions = static_cast<int32_t*>(a.array(at + 2, ScalarType::Int, {g->axes, t}, idx));
  }
  g->pairs = a.tensor(at + 3).numel();
  if (g->pairs > FP8BL_MAX_PAIRS)
    value_error("at most " + std::to_string(FP8BL_MAX_PAIRS) + " pairs, got " + std::to_string(g->pairs));
  g->inv_freq = static_cast<float*>(a.array(at + 3, ScalarType::Float, {g->pairs}, idx));
  if (!a.given(how)) {
    if (g->axes != 1) value_error("axes is needed where positions has several");
  } else {
    const auto wrong = [&](Py_ssize_t n) {
      value_error("axes names " + std::to_string(n) + " pairs, inv_freq has " + std::to_string(g->pairs));
    };
    if (PyBytes_Check(a.v[how])) {
      const Py_ssize_t n = PyBytes_GET_SIZE(a.v[how]);
      if (n != g->pairs) wrong(n);
      for (Py_ssize_t i = 0; i < n; ++i) g->axis[i] = (uint8_t)PyBytes_AS_STRING(a.v[how])[i];
    } else {
      PyObject* seq = PySequence_Fast(a.v[how], "axes must be a sequence of axis numbers");
      if (!seq) throw Raise{nullptr, {}};
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      bool ok = n == g->pairs;
      for (Py_ssize_t i = 0; ok && i < n; ++i) {
        const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
        if (v < 0 || v > 255) {
          Py_DECREF(seq);
          if (PyErr_Occurred()) throw Raise{nullptr, {}};
          value_error("axes must be axis numbers");
        }
        g->axis[i] = (uint8_t)v;
      }
      Py_DECREF(seq);
      if (!ok) wrong(n);
    }
  }
  g->eps = a.number(how + 1, 1e-6);
  g->interleaved = a.truth(how + 2, false);
}

// The cache: parameters `at` .. at + 4 are k_cache, v_cache, k_scale and v_scale;
// `slots` is the parameter of the slots.
void set_cache(const Args& a, int slots, int at, int64_t idx, fp8bl_qkv* g) {
  g->cache_rows = a.head_shape(at)[0];
  const int64_t r = g->cache_rows, h = g->k_heads, d = g->head_dim;
  g->slots = static_cast<int32_t*>(a.array(slots, ScalarType::Int, {g->tokens}, idx));
  g->k_cache = static_cast<uint8_t*>(a.array(at, ScalarType::Byte, {r, h, d}, idx));
  g->v_cache = static_cast<uint8_t*>(a.array(at + 1, ScalarType::Byte, {r, h, d}, idx));
  g->k_scale = static_cast<float*>(a.array(at + 2, ScalarType::Float, {r, h}, idx));
  g->v_scale = static_cast<float*>(a.array(at + 3, ScalarType::Float, {r, h}, idx));
}

// The cache was written: parameters as above.
void cache_written(const Args& a, int at) {
  for (int i = 0; i < 4; ++i) written(a.tensor(at + i));
}

// Sizes from the parameters that hold q and k.
fp8bl_qkv sizes(const Args& a, int q, int k) {
  fp8bl_qkv g{};
  const at::IntArrayRef qs = a.head_shape(q), ks = a.head_shape(k);
  g.tokens = qs[0];
  g.q_heads = qs[1];
  g.k_heads = ks[1];
  g.head_dim = qs[2];
  return g;
}

Signature kNormRope{"fp8_qk_norm_rope", 6, 11,
                    {"q", "k", "q_weight", "k_weight", "positions", "inv_freq", "axes", "eps", "interleaved", "q_out",
                     "k_out"},
                    "fp8_qk_norm_rope_backward"};
PyObject* norm_rope(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& q = a.tensor(0);
  const c10::DeviceGuard guard(q.device());
  fp8bl_qkv g = sizes(a, 0, 1);
  const int64_t qs[] = {g.tokens, g.q_heads, g.head_dim}, ks[] = {g.tokens, g.k_heads, g.head_dim};
  g.q = a.heads(0, qs, idx);
  g.k = a.heads(1, ks, idx);
  set_turn(a, 2, 6, idx, &g);
  Output qo(a, 9, qs, ScalarType::BFloat16, q), ko(a, 10, ks, ScalarType::BFloat16, q);
  const With wq(a, 9, qo), wk(a, 10, ko);
  g.q_out = a.heads(9, qs, idx);
  g.k_out = a.heads(10, ks, idx);
  const hipStream_t st = stream_of(idx);
  run("fp8_qk_norm_rope", [&] { return fp8_qk_norm_rope(&g, st); });
  return pair(qo, ko);
}

Signature kNormRopeBackward{"fp8_qk_norm_rope_backward", 8, 15,
                            {"dq", "dk", "q", "k", "q_weight", "k_weight", "positions", "inv_freq", "axes", "eps",
                             "interleaved", "q_grad", "k_grad", "need_weights", "workspace"}};
PyObject* norm_rope_backward(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(2);
  const Tensor& q = a.tensor(2);
  const c10::DeviceGuard guard(q.device());
  fp8bl_qkv g = sizes(a, 2, 3);
  const int64_t qs[] = {g.tokens, g.q_heads, g.head_dim}, ks[] = {g.tokens, g.k_heads, g.head_dim};
  g.dq = a.heads(0, qs, idx);
  g.dk = a.heads(1, ks, idx);
  g.q = a.heads(2, qs, idx);
  g.k = a.heads(3, ks, idx);
  set_turn(a, 4, 8, idx, &g);
  Output qg(a, 11, qs, ScalarType::BFloat16, q), kg(a, 12, ks, ScalarType::BFloat16, q);
  const With wq(a, 11, qg), wk(a, 12, kg);
  g.q_out = a.heads(11, qs, idx);
  g.k_out = a.heads(12, ks, idx);
  PyObject* weights[2] = {nullptr, nullptr};
  const bool need = a.truth(13, true);
  Tensor dqw, dkw;
  if (need) {
    dqw = fresh({g.head_dim}, ScalarType::Float, q);
    dkw = fresh({g.head_dim}, ScalarType::Float, q);
    g.dq_weight = static_cast<float*>(dqw.data_ptr());
    g.dk_weight = static_cast<float*>(dkw.data_ptr());
  }
  const Workspace w(a, 14, fp8_qk_norm_rope_backward_workspace_size(g.tokens, g.q_heads, g.k_heads, g.head_dim), idx, q);
  const hipStream_t st = stream_of(idx);
  run("fp8_qk_norm_rope_backward", [&] { return fp8_qk_norm_rope_backward(&g, w.p, w.bytes, st); });
  if (need) {
    weights[0] = THPVariable_Wrap(dqw);
    weights[1] = THPVariable_Wrap(dkw);
  }
  PyObject* t = PyTuple_New(4);
  if (!t || (need && (!weights[0] || !weights[1]))) {
    Py_XDECREF(t);
    Py_XDECREF(weights[0]);
    Py_XDECREF(weights[1]);
    throw Raise{nullptr, {}};
  }
  PyTuple_SET_ITEM(t, 0, qg.release());
  PyTuple_SET_ITEM(t, 1, kg.release());
  for (int i = 0; i < 2; ++i) {
    if (!need) {
      weights[i] = Py_None;
      Py_INCREF(Py_None);
    }
    PyTuple_SET_ITEM(t, 2 + i, weights[i]);
  }
  return t;
}

Signature kStore{"fp8_kv_store", 7, 7, {"k", "v", "slots", "k_cache", "v_cache", "k_scale", "v_scale"}};
PyObject* store(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const c10::DeviceGuard guard(a.tensor(0).device());
  fp8bl_qkv g = sizes(a, 0, 0);
  const int64_t ks[] = {g.tokens, g.k_heads, g.head_dim};
  g.q_heads = 0;
  g.k = a.heads(0, ks, idx);
  g.v = a.heads(1, ks, idx);
  set_cache(a, 2, 3, idx, &g);
  const hipStream_t st = stream_of(idx);
  run("fp8_kv_store", [&] { return fp8_kv_store(&g, st); });
  cache_written(a, 3);
  Py_RETURN_NONE;
}

Signature kLoad{"fp8_kv_load", 5, 7, {"k_cache", "v_cache", "k_scale", "v_scale", "slots", "k_out", "v_out"}};
PyObject* load(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& c = a.tensor(0);
  const c10::DeviceGuard guard(c.device());
  fp8bl_qkv g = sizes(a, 0, 0);
  g.tokens = a.tensor(4).numel();
  g.q_heads = 0;
  set_cache(a, 4, 0, idx, &g);
  const int64_t ks[] = {g.tokens, g.k_heads, g.head_dim};
  Output k(a, 5, ks, ScalarType::BFloat16, c), v(a, 6, ks, ScalarType::BFloat16, c);
  const With wk(a, 5, k), wv(a, 6, v);
  g.k_out = a.heads(5, ks, idx);
  g.v_out = a.heads(6, ks, idx);
  const hipStream_t st = stream_of(idx);
  run("fp8_kv_load", [&] { return fp8_kv_load(&g, st); });
  return pair(k, v);
}

Signature kNormRopeStore{"fp8_qk_norm_rope_store", 12, 16,
                         {"q", "k", "v", "q_weight", "k_weight", "positions", "inv_freq", "slots", "k_cache", "v_cache",
                          "k_scale", "v_scale", "axes", "eps", "interleaved", "q_out"}};
PyObject* norm_rope_store(Args a) {
  a.outside_autograd();
  const int64_t idx = a.device(0);
  const Tensor& q = a.tensor(0);
  const c10::DeviceGuard guard(q.device());
  fp8bl_qkv g = sizes(a, 0, 1);
  const int64_t qs[] = {g.tokens, g.q_heads, g.head_dim}, ks[] = {g.tokens, g.k_heads, g.head_dim};
  g.q = a.heads(0, qs, idx);
  g.k = a.heads(1, ks, idx);
  g.v = a.heads(2, ks, idx);
  set_turn(a, 3, 12, idx, &g);
  set_cache(a, 7, 8, idx, &g);
  Output qo(a, 15, qs, ScalarType::BFloat16, q);
  const With wq(a, 15, qo);
  g.q_out = a.heads(15, qs, idx);
  const hipStream_t st = stream_of(idx);
  run("fp8_qk_norm_rope_store", [&] { return fp8_qk_norm_rope_store(&g, st); });
  cache_written(a, 8);
  return qo.release();
}

// ---- The module.

template <Signature& S, PyObject* (*F)(Args)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n, PyObject* names) {
  try {
    return F(Args(S, args, n, names));
  } catch (const Raise& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_memory, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// configure(error class, raw stream function, out-of-memory error class)
PyObject* configure(PyObject*, PyObject* args) {
  PyObject* given[3];
  if (!PyArg_ParseTuple(args, "OOO", &given[0], &given[1], &given[2])) return nullptr;
  PyObject** const kept[] = {&g_error, &g_raw_stream, &g_memory};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(given[i]);
    PyObject* const was = *kept[i];
    *kept[i] = given[i];
    Py_XDECREF(was);
  }
  Py_RETURN_NONE;
}

#define FUNCTION(sig, fn, doc) \
  {sig.name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<sig, fn>)), METH_FASTCALL | METH_KEYWORDS, doc}

PyMethodDef kFunctions[] = {
    FUNCTION(kRowQuantize, row_quantize,
             "int8_row_quantize(x, q=None, scale=None)\n--\n\n"
             "fp32 or bf16 x [M,K] -> (q int8 [M,K], scale fp32 [M]), x ~ q * scale: the\n"
             "tokens of an activation or the output channels of a weight [N,K]."),
    FUNCTION(kLinear, linear,
             "int8_linear(xq, x_scale, wq, w_scale, bias=None, out=None, workspace=None)\n--\n\n"
             "int8 xq [M,K] with x_scale [M], int8 wq [N,K] with w_scale [N] -> bf16\n"
             "y [M,N] = (xq wq^T) x_scale w_scale + bias, the integer sum exact.\n\n"
             "bias bf16 [N]. workspace, when given, holds at least\n"
             "int8_workspace_size(M, N, K, from_bf16=False) bytes; calls that share one\n"
             "must be ordered."),
    FUNCTION(kLinearBf16, linear_bf16,
             "int8_linear_bf16(x, wq, w_scale, bias=None, out=None, workspace=None)\n--\n\n"
             "bf16 x [M,K] -> int8_row_quantize -> int8_linear, the same bits as those two\n"
             "calls. workspace, when given, holds at least int8_workspace_size(M, N, K)\n"
             "bytes; calls that share one must be ordered."),
    FUNCTION(kNormRope, norm_rope,
             "fp8_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, axes=None, eps=1e-6,\n"
             "                 interleaved=False, q_out=None, k_out=None)\n--\n\n"
             "Norm and rotation of each head of bf16 q [T,Hq,D] and k [T,Hk,D] -> (q_out, k_out):\n"
             "x / sqrt(mean(x^2) + eps) * weight, then pair i turned by\n"
             "positions[axes[i], token] * inv_freq[i].\n\n"
             "q and k may be views of the projection's output (last axis contiguous, the\n"
             "other strides multiples of 8); q_out may be q and k_out k. Weights bf16 [D];\n"
             "positions int32 [axes, T] or [T]; inv_freq fp32 [P]; axes a sequence of P axis\n"
             "numbers on the host (a tuple or bytes), not needed with one axis. Pair i is\n"
             "elements (i, i + P), or (2 i, 2 i + 1) with interleaved; elements from 2 P on are\n"
             "not turned. D is a multiple of 8 from 16 to 256, P of 8 (4 with interleaved).\n\n"
             "Not recorded by autograd: while gradients are enabled, tensors that require one\n"
             "are refused; fp8_qk_norm_rope_backward is its backward pass."),
    FUNCTION(kNormRopeBackward, norm_rope_backward,
             "fp8_qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, axes=None,\n"
             "                          eps=1e-6, interleaved=False, q_grad=None, k_grad=None,\n"
             "                          need_weights=True, workspace=None)\n--\n\n"
             "Backward pass of fp8_qk_norm_rope: the gradients dq, dk of what it returned and its\n"
             "own inputs -> (q_grad, k_grad, q_weight_grad, k_weight_grad), the first two bf16\n"
             "like q and k (they may be given, as views of one packed gradient, or as dq and dk\n"
             "themselves), the others fp32 [D], None with need_weights false. workspace, when\n"
             "given, holds at least qk_norm_rope_backward_workspace_size(T, Hq, Hk, D) bytes."),
    FUNCTION(kStore, store,
             "fp8_kv_store(k, v, slots, k_cache, v_cache, k_scale, v_scale)\n--\n\n"
             "bf16 k and v [T,H,D] into rows slots (int32 [T]) of an E4M3 cache: codes uint8\n"
             "[rows,H,D] with a scale fp32 [rows,H] for each token and head, S = amax / 448.\n\n"
             "A token whose slot is negative or past the cache is padding and not stored; where\n"
             "tokens share a slot the last one is. Pages are rows too: slot = page * page size +\n"
             "offset, for caches viewed as [rows,H,D]. At most 65536 tokens a call."),
    FUNCTION(kLoad, load,
             "fp8_kv_load(k_cache, v_cache, k_scale, v_scale, slots, k_out=None, v_out=None)\n--\n\n"
             "Rows slots (int32 [T]) of the cache -> (k, v) bf16 [T,H,D], zeros for a slot\n"
             "outside the cache. k_out and v_out may be views with strides."),
    FUNCTION(kNormRopeStore, norm_rope_store,
             "fp8_qk_norm_rope_store(q, k, v, q_weight, k_weight, positions, inv_freq, slots, k_cache,\n"
             "                       v_cache, k_scale, v_scale, axes=None, eps=1e-6, interleaved=False,\n"
             "                       q_out=None)\n--\n\n"
             "fp8_qk_norm_rope and fp8_kv_store in one pass -> q_out: the cache receives v and the\n"
             "normed and turned k, quantized from fp64 (storing a returned k rounds it to bf16\n"
             "first)."),
    {"configure", configure, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, kFunctions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() {
  for (Signature* s : {&kRowQuantize, &kLinear, &kLinearBf16, &kNormRope, &kNormRopeBackward, &kStore, &kLoad,
                       &kNormRopeStore})
    for (int i = 0; i < s->count; ++i)
      if (!(s->interned[i] = PyUnicode_InternFromString(s->params[i]))) return nullptr;
  return PyModule_Create(&kModule);
}
