// zc_torch.cpp -- Python entry points of the operators around an expert-parallel exchange and of the
// training step around it (moe.py, norm.py, dropout.py, embedding.py): torch tensors in, checked, outputs
// allocated by torch, and one call of the C ABI (include/zc.h) on the current torch stream or the one
// given.  Argument marshalling only, as zc.py
// does with ctypes; native because these operators run for a few microseconds in a decoding step,
// where five allocations, a dozen attributes and a ctypes call in Python cost more than the kernels
// (route of 8 tokens: 9.5 us of host time in Python).
//
// Errors: a wrong tensor raises ValueError, an error of the C ABI zc.ZcError, torch's own errors
// (out of memory) as torch raises them.
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>

#include "zc.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // zc.ZcError

// Unwinds to the entry point with a Python exception set.
struct Raised {};

[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(PyExc_ValueError, why.c_str());
  throw Raised();
}

void check(zc_status s, const char* where) {
  if (s == ZC_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(s), where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); i++) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// A torch.Tensor or of a class derived from it (isinstance() would ask the metaclass, 0.1 us a float).
bool is_tensor(PyObject* o) { return PyObject_TypeCheck(o, reinterpret_cast<PyTypeObject*>(THPVariableClass)); }

const Tensor& tensor(PyObject* o, const char* what) {
  if (!is_tensor(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}

// The kernels read and write all of a call's tensors on one device (checked before anything else).
void one_device(PyObject* const* args, Py_ssize_t n) {
  const Tensor* first = nullptr;
  for (Py_ssize_t i = 0; i < n; i++) {
    if (!is_tensor(args[i])) continue;
    const Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda()) refuse("libzc takes CUDA tensors");
    if (!first)
      first = &t;
    else if (t.device() != first->device())
      refuse("the tensors are on more than one device: " + first->device().str() + " and " + t.device().str());
  }
}

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return ZC_BF16;
    case at::kHalf: return ZC_F16;
    case at::kFloat: return ZC_F32;
    default: refuse("activations are bfloat16, float16 or float32");
  }
}

// An input matrix: contiguous columns, rows `stride` values apart.
struct Matrix {
  const Tensor& t;
  uint64_t rows, width, stride;
  const void* p() const { return t.const_data_ptr(); }
};

Matrix matrix(PyObject* o, const char* what) {
  const Tensor& t = tensor(o, what);
  if (t.dim() != 2) refuse(std::string(what) + " must be a matrix (rows, width), not " + shape_of(t));
  const bool none = t.size(0) == 0;  // of no rows the strides are anything
  if (t.stride(1) != 1 && t.size(1) > 1 && !none) refuse(std::string(what) + " must have contiguous columns");
  return {t, static_cast<uint64_t>(t.size(0)), static_cast<uint64_t>(t.size(1)),
          static_cast<uint64_t>(none ? t.size(1) : t.stride(0))};
}

Matrix same_as(PyObject* o, const Tensor& like, const char* what) {
  const Matrix m = matrix(o, what);
  if (m.t.sizes() != like.sizes() || m.t.scalar_type() != like.scalar_type())
    refuse(std::string(what) + " must have the shape and type of the activations");
  return m;
}

// A contiguous table of a given type and shape.
const Tensor& table(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* what) {
  const Tensor& t = tensor(o, what);
  if (t.scalar_type() != type || t.sizes() != shape)
    refuse(std::string(what) + " has the wrong type or shape " + shape_of(t));
  if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
  return t;
}

int score_of(PyObject* o) {
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (s && std::string(s) == "softmax") return ZC_SOFTMAX;
  if (s && std::string(s) == "sigmoid") return ZC_SIGMOID;
  refuse("score must be 'softmax' or 'sigmoid'");
}

long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();  // an array of several values, say
  return v != 0;
}

// A count that the C ABI takes as 32 bits; what it refuses as too large stays so.
uint32_t count(PyObject* o, const char* what) {
  const long v = integer(o);
  if (v < 0) refuse(std::string(what) + " must not be negative");
  return v > 0x7FFFFFFFl ? 0x7FFFFFFFu : static_cast<uint32_t>(v);
}

// A size that the C ABI takes as 32 bits and refuses as too large from 2^31 on.
uint32_t narrow(uint64_t size, const char* where) {
  if (size > 0x7FFFFFFFull) check(ZC_ERR_TOO_LARGE, where);
  return static_cast<uint32_t>(size);
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(v);
}

// Where a call launches: on the activations' device, which is the current one while the call lasts,
// and there on the given torch stream, else on the current one.  Its outputs come from the
// allocator for that stream, for a block is only safe to write on the stream that it was last used
// on: a given stream is the current one while the call lasts.  What it makes there is also recorded
// on the stream that was current before, so that the caller may use and drop it on either (once
// ordered behind the launch).
class Launch {
 public:
  Launch(PyObject* stream, const Tensor& like) : device_(like.device()) {
    if (c10::cuda::current_device() != device_.index()) current_.set_device(device_);
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(device_.index());
    stream_ = current.stream();
    if (stream == Py_None) return;
    PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
    if (!raw) throw Raised();
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (PyErr_Occurred()) throw Raised();
    PyObject* index = PyObject_GetAttrString(stream, "device_index");
    if (!index) PyErr_Clear();  // a handle alone
    const long on = index ? PyLong_AsLong(index) : device_.index();
    Py_XDECREF(index);
    if (PyErr_Occurred()) throw Raised();
    if (on != device_.index()) refuse("the stream is on another device than the tensors");
    if (s == stream_) return;
    stream_ = s;
    caller_ = current;
    given_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), device_.index()));
  }

  void* stream() const { return stream_; }

  // A new tensor, straight from torch's allocator of device memory: the way there through torch's
  // dispatcher takes 0.25 us more (a dispatch of 8 tokens 7.8 us of host time instead of 6.8).
  Tensor fresh(at::IntArrayRef shape, at::ScalarType type) const {
    return kept(at::detail::empty_cuda(shape, type, device_, std::nullopt));
  }
  Tensor zeros(at::IntArrayRef shape, at::ScalarType type) const {
    return kept(at::zeros(shape, at::TensorOptions(type).device(device_)));
  }
  // The caller's output tensor, checked, or a new one.
  Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const char* what) const {
    if (o == Py_None) return fresh(shape, type);
    return table(o, shape, type, what);
  }

 private:
  Tensor kept(Tensor t) const {
    if (caller_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *caller_);
    return t;
  }

  c10::Device device_;
  c10::cuda::OptionalCUDAGuard current_;
  void* stream_;
  std::optional<c10::cuda::CUDAStream> caller_;  // with a given stream: the current one before
  std::optional<c10::cuda::CUDAStreamGuard> given_;
};

PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined())
      o = THPVariable_Wrap(t);
    else
      Py_INCREF(o);
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <typename F>
zc_status without_gil(F&& f) {
  zc_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

using Args = PyObject* const*;

// (logits, k, score, bias, renormalize, scale, weights, experts, stream) -> (weights, experts)
PyObject* moe_route(Args a) {
  const Matrix l = matrix(a[0], "logits");
  const int64_t tokens = l.t.size(0);
  const uint32_t k = count(a[1], "k");
  const int dtype = dtype_of(l.t), score = score_of(a[2]), renormalize = truth(a[4]);
  const float* bias = nullptr;
  if (a[3] != Py_None) bias = static_cast<const float*>(table(a[3], {l.t.size(1)}, at::kFloat, "bias").const_data_ptr());
  const float scale = real(a[5]);
  const uint32_t width = narrow(l.width, "zc_moe_route");
  if (k > ZC_MOE_MAX_K) check(ZC_ERR_TOO_LARGE, "zc_moe_route");  // before outputs of that size are made
  const Launch on(a[8], l.t);
  Tensor weights = on.output(a[6], {tokens, k}, at::kFloat, "weights");
  Tensor experts = on.output(a[7], {tokens, k}, at::kInt, "experts");
  check(without_gil([&] {
          return zc_moe_route(l.p(), dtype, l.stride, l.rows, width, k, score, bias, renormalize, scale,
                              static_cast<float*>(weights.mutable_data_ptr()),
                              static_cast<int32_t*>(experts.mutable_data_ptr()), on.stream());
        }),
        "zc_moe_route");
  return pack({weights, experts});
}

// (dweights, logits, experts, score, renormalize, scale, dlogits, stream) -> (dlogits,)
PyObject* moe_route_backward(Args a) {
  const Matrix l = matrix(a[1], "logits");
  const Tensor& experts = tensor(a[2], "experts");
  if (experts.dim() != 2) refuse("experts must be [tokens, k]");
  const int64_t tokens = l.t.size(0), k = experts.size(1);
  table(a[2], {tokens, k}, at::kInt, "experts");
  const Tensor& dweights = table(a[0], {tokens, k}, at::kFloat, "dweights");
  const int dtype = dtype_of(l.t), score = score_of(a[3]), renormalize = truth(a[4]);
  const float scale = real(a[5]);
  const uint32_t width = narrow(l.width, "zc_moe_route_backward");
  const uint32_t slots = narrow(static_cast<uint64_t>(k), "zc_moe_route_backward");
  const Launch on(a[7], l.t);
  Tensor dlogits = on.output(a[6], l.t.sizes(), l.t.scalar_type(), "dlogits");
  check(without_gil([&] {
          return zc_moe_route_backward(static_cast<const float*>(dweights.const_data_ptr()), l.p(), dtype, l.stride,
                                       l.rows, width, slots,
                                       static_cast<const int32_t*>(experts.const_data_ptr()), score, renormalize,
                                       scale, dlogits.mutable_data_ptr(), on.stream());
        }),
        "zc_moe_route_backward");
  return pack({dlogits});
}

// (x, experts, num_experts, ws, rows, stream) -> (rows, positions, slots, offsets)
PyObject* moe_dispatch(Args a) {
  const Matrix x = matrix(a[0], "x");
  const Tensor& experts = tensor(a[1], "experts");
  const int64_t tokens = x.t.size(0);
  if (experts.dim() != 2 || experts.size(0) != tokens ||
      (experts.scalar_type() != at::kInt && experts.scalar_type() != at::kLong))
    refuse("experts must be int32 or int64 [tokens, k]");
  if (!experts.is_contiguous()) refuse("libzc takes contiguous tensors");
  const int64_t k = experts.size(1);
  const uint32_t n = count(a[2], "num_experts");
  const Tensor& ws = tensor(a[3], "ws");
  if (!ws.is_contiguous()) refuse("libzc takes contiguous tensors");
  const int dtype = dtype_of(x.t);
  const uint32_t hidden = narrow(x.width, "zc_moe_dispatch");
  if (n > ZC_MOE_MAX_EXPERTS || k > ZC_MOE_MAX_K) check(ZC_ERR_TOO_LARGE, "zc_moe_dispatch");
  const Launch on(a[5], x.t);
  Tensor rows = on.output(a[4], {tokens * k, x.t.size(1)}, x.t.scalar_type(), "rows");
  Tensor positions = on.fresh({tokens, k}, at::kInt), slots = on.fresh({tokens * k}, at::kInt);
  Tensor offsets = on.fresh({static_cast<int64_t>(n) + 1}, at::kInt);
  check(without_gil([&] {
          return zc_moe_dispatch(x.p(), dtype, x.stride, x.rows, hidden, experts.const_data_ptr(),
                                 experts.scalar_type() == at::kLong, static_cast<uint32_t>(k), n,
                                 rows.mutable_data_ptr(), static_cast<int32_t*>(positions.mutable_data_ptr()),
                                 static_cast<int32_t*>(slots.mutable_data_ptr()),
                                 static_cast<int32_t*>(offsets.mutable_data_ptr()), ws.mutable_data_ptr(),
                                 static_cast<uint64_t>(ws.nbytes()), on.stream());
        }),
        "zc_moe_dispatch");
  return pack({rows, positions, slots, offsets});
}

const Tensor& positions_of(PyObject* o) {
  const Tensor& t = tensor(o, "positions");
  if (t.dim() != 2 || t.scalar_type() != at::kInt) refuse("positions must be int32 [tokens, k]");
  if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
  return t;
}

// (rows, weights or None, positions, status, out, stream) -> (out,)
PyObject* moe_combine(Args a) {
  const Matrix r = matrix(a[0], "rows");
  const Tensor& positions = positions_of(a[2]);
  const int64_t tokens = positions.size(0), k = positions.size(1);
  const int dtype = dtype_of(r.t);
  const uint32_t hidden = narrow(r.width, "zc_moe_combine"), slots = narrow(static_cast<uint64_t>(k), "zc_moe_combine");
  const float* weights = nullptr;
  if (a[1] != Py_None)
    weights = static_cast<const float*>(table(a[1], {tokens, k}, at::kFloat, "weights").const_data_ptr());
  const Tensor& status = table(a[3], {1}, at::kInt, "status");
  const Launch on(a[5], r.t);
  Tensor out = on.output(a[4], {tokens, r.t.size(1)}, r.t.scalar_type(), "out");
  check(without_gil([&] {
          return zc_moe_combine(r.p(), dtype, r.stride, r.rows, weights,
                                static_cast<const int32_t*>(positions.const_data_ptr()),
                                static_cast<uint64_t>(tokens), slots, hidden, out.mutable_data_ptr(),
                                static_cast<int32_t*>(status.mutable_data_ptr()), on.stream());
        }),
        "zc_moe_combine");
  return pack({out});
}

// (dout, rows, weights, positions, status, drows, dweights, stream) -> (drows, dweights)
PyObject* moe_combine_backward(Args a) {
  const Matrix r = matrix(a[1], "rows"), g = matrix(a[0], "dout");
  const Tensor& positions = positions_of(a[3]);
  const int64_t tokens = positions.size(0), k = positions.size(1);
  if (g.t.scalar_type() != r.t.scalar_type() || g.t.size(0) != tokens || g.width != r.width)
    refuse("dout must be [tokens, hidden] in the rows' type");
  const int dtype = dtype_of(r.t);
  const uint32_t hidden = narrow(r.width, "zc_moe_combine_backward");
  const uint32_t slots = narrow(static_cast<uint64_t>(k), "zc_moe_combine_backward");
  const Tensor& weights = table(a[2], {tokens, k}, at::kFloat, "weights");
  const Tensor& status = table(a[4], {1}, at::kInt, "status");
  const Launch on(a[7], r.t);
  Tensor drows = on.output(a[5], r.t.sizes(), r.t.scalar_type(), "drows");
  Tensor dweights = on.output(a[6], {tokens, k}, at::kFloat, "dweights");
  check(without_gil([&] {
          return zc_moe_combine_backward(
              g.p(), dtype, g.stride, r.p(), r.stride, r.rows, static_cast<const float*>(weights.const_data_ptr()),
              static_cast<const int32_t*>(positions.const_data_ptr()), static_cast<uint64_t>(tokens),
              slots, hidden, drows.mutable_data_ptr(), static_cast<float*>(dweights.mutable_data_ptr()),
              static_cast<int32_t*>(status.mutable_data_ptr()), on.stream());
        }),
        "zc_moe_combine_backward");
  return pack({drows, dweights});
}

// Fills in the parameters that zc_norm_args and zc_norm_backward_args share.
template <typename A>
void norm_params(A& a, const Tensor& x, PyObject* weight, PyObject* gate, PyObject* next_weight) {
  a.tokens = static_cast<uint64_t>(x.size(0));
  a.hidden = x.size(1) > 0x7FFFFFFF ? 0x7FFFFFFFu : static_cast<uint32_t>(x.size(1));
  a.dtype = dtype_of(x);
  bool first = true;
  at::ScalarType kind = x.scalar_type();
  auto param = [&](PyObject* o, const char* what) -> const Tensor& {
    const Tensor& t = tensor(o, what);
    if (first) kind = t.scalar_type();
    first = false;
    if (t.scalar_type() != kind || (kind != x.scalar_type() && kind != at::kFloat))
      refuse("weights and gate must all have the activations' type, or all be float32");
    if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
    return t;
  };
  auto vector = [&](PyObject* o, const char* what) -> const void* {
    if (o == Py_None) return nullptr;
    const Tensor& t = param(o, what);
    if (t.dim() != 1 || t.size(0) != x.size(1))
      refuse(std::string(what) + " must have the activations' width, not " + shape_of(t));
    return t.const_data_ptr();
  };
  a.weight = vector(weight, "weight");
  a.next_weight = vector(next_weight, "next_weight");
  if (gate != Py_None) {
    const Tensor& g = param(gate, "gate");
    if (g.dim() != 2 || (g.size(1) != 1 && g.size(1) != x.size(1)) || g.size(0) < 1 || x.size(0) % g.size(0))
      refuse("gate must be [rows, hidden] or [rows, 1] with rows a divisor of the tokens");
    a.gate = g.const_data_ptr();
    a.gate_rows = static_cast<uint64_t>(g.size(0));
    a.gate_wide = g.size(1) == x.size(1);
  }
  a.params_f32 = kind == at::kFloat && x.scalar_type() != at::kFloat;
}

// (y or None, x, weight, gate, residual_scale, next_weight, eps, x_new, h, stream) -> (x_new or
// None, h or None)
PyObject* norm_forward(Args a) {
  zc_norm_args n = {};
  const bool branch = a[0] != Py_None;
  const Matrix x = matrix(a[1], "x");
  if (branch) {
    const Matrix y = same_as(a[0], x.t, "y");
    n.y = y.p();
    n.y_stride = y.stride;
    if (a[2] == Py_None) refuse("the norm after a block takes a weight");
  }
  n.x = x.p();
  n.x_stride = x.stride;
  norm_params(n, x.t, a[2], a[3], a[5]);
  n.residual_scale = real(a[4]);
  n.eps = real(a[6]);
  const Launch on(a[9], x.t);
  Tensor x_new, h;
  if (branch) x_new = on.output(a[7], x.t.sizes(), x.t.scalar_type(), "x_new");
  if (a[5] != Py_None) h = on.output(a[8], x.t.sizes(), x.t.scalar_type(), branch ? "h" : "out");
  if (x_new.defined()) n.x_new = x_new.mutable_data_ptr();
  if (h.defined()) n.h = h.mutable_data_ptr();
  check(without_gil([&] { return zc_norm(&n, on.stream()); }), "zc_norm");
  return pack({x_new, h});
}

// (dx_new, dh, y, x_new, weight, gate, residual_scale, next_weight, eps, ws, stream; any of the
// first four may be None) -> (dy, dx, dweight, dgate, dnext_weight)
PyObject* norm_backward(Args a) {
  zc_norm_backward_args n = {};
  const bool branch = a[2] != Py_None;
  const Matrix like = matrix(branch ? a[2] : a[3], branch ? "y" : "x");
  const Tensor& x = like.t;
  if (branch) {
    n.y = like.p();
    n.y_stride = like.stride;
  }
  if (a[0] != Py_None) {
    const Matrix m = same_as(a[0], x, "dx_new");
    n.dx_new = m.p();
    n.dx_new_stride = m.stride;
  }
  if (a[1] != Py_None) {
    const Matrix m = same_as(a[1], x, "dh");
    n.dh = m.p();
    n.dh_stride = m.stride;
  }
  if (a[3] != Py_None && a[7] != Py_None) {
    const Matrix m = same_as(a[3], x, "x_new");
    n.x_new = m.p();
    n.x_new_stride = m.stride;
  }
  norm_params(n, x, a[4], a[5], a[7]);
  n.residual_scale = real(a[6]);
  n.eps = real(a[8]);
  const bool none = x.size(0) == 0;  // no tokens: nothing to launch, and the sums over none of them are zero
  const Launch on(a[10], x);
  Tensor dy, dx = on.fresh(x.sizes(), x.scalar_type()), grads[3];
  if (branch) dy = on.fresh(x.sizes(), x.scalar_type());
  for (int i = 0; i < 3; i++) {
    PyObject* o = a[i == 0 ? 4 : i == 1 ? 5 : 7];
    if (o == Py_None) continue;
    const Tensor& p = THPVariable_Unpack(o);
    grads[i] = none ? on.zeros(p.sizes(), p.scalar_type()) : on.fresh(p.sizes(), p.scalar_type());
  }
  if (!none) {
    const Tensor& ws = tensor(a[9], "ws");
    if (!ws.is_contiguous()) refuse("libzc takes contiguous tensors");
    n.dx = dx.mutable_data_ptr();
    if (dy.defined()) n.dy = dy.mutable_data_ptr();
    if (grads[0].defined()) n.dweight = grads[0].mutable_data_ptr();
    if (grads[1].defined()) n.dgate = grads[1].mutable_data_ptr();
    if (grads[2].defined()) n.dnext_weight = grads[2].mutable_data_ptr();
    n.ws = ws.mutable_data_ptr();
    n.ws_bytes = static_cast<uint64_t>(ws.nbytes());
    check(without_gil([&] { return zc_norm_backward(&n, on.stream()); }), "zc_norm_backward");
  }
  return pack({dy, dx, grads[0], grads[1], grads[2]});
}

// A mask of one byte a token, or NULL.
const uint8_t* mask_of(PyObject* o, int64_t tokens) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, "mask");
  if ((t.scalar_type() != at::kBool && t.scalar_type() != at::kByte) || t.dim() != 1 || t.size(0) != tokens)
    refuse("mask must be bool or uint8 [tokens], not " + shape_of(t));
  if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
  return static_cast<const uint8_t*>(t.const_data_ptr());
}

// (logits, experts, ws, score, sequences, mask, stream) -> (loss, counts, slope)
PyObject* moe_balance(Args a) {
  const Matrix l = matrix(a[0], "logits");
  const Tensor& experts = tensor(a[1], "experts");
  const int64_t tokens = l.t.size(0), width = l.t.size(1);
  if (experts.dim() != 2) refuse("experts must be [tokens, k]");
  const int64_t k = experts.size(1);
  table(a[1], {tokens, k}, at::kInt, "experts");
  const Tensor& ws = tensor(a[2], "ws");
  if (!ws.is_contiguous()) refuse("libzc takes contiguous tensors");
  const int dtype = dtype_of(l.t), score = score_of(a[3]);
  const int64_t sequences = integer(a[4]);
  if (sequences < 1 || tokens % sequences) refuse("sequences must be a divisor of the tokens");
  const uint8_t* mask = mask_of(a[5], tokens);
  const uint32_t n = narrow(l.width, "zc_moe_balance"), slots = narrow(static_cast<uint64_t>(k), "zc_moe_balance");
  if (n > ZC_MOE_MAX_EXPERTS || sequences > 0x7FFFFFFF) check(ZC_ERR_TOO_LARGE, "zc_moe_balance");
  const Launch on(a[6], l.t);
  Tensor loss = on.fresh({}, at::kFloat), counts = on.fresh({sequences, width}, at::kInt);
  Tensor slope = on.fresh({sequences, width}, at::kFloat);
  check(without_gil([&] {
          return zc_moe_balance(l.p(), dtype, l.stride, l.rows, n, slots,
                                static_cast<const int32_t*>(experts.const_data_ptr()), score,
                                static_cast<uint64_t>(sequences), mask, static_cast<float*>(loss.mutable_data_ptr()),
                                static_cast<int32_t*>(counts.mutable_data_ptr()),
                                static_cast<float*>(slope.mutable_data_ptr()), ws.mutable_data_ptr(),
                                static_cast<uint64_t>(ws.nbytes()), on.stream());
        }),
        "zc_moe_balance");
  return pack({loss, counts, slope});
}

// (dloss, logits, slope, score, mask, dlogits, stream) -> (dlogits,)
PyObject* moe_balance_backward(Args a) {
  const Matrix l = matrix(a[1], "logits");
  const Tensor& dloss = tensor(a[0], "dloss");
  if (dloss.numel() != 1 || dloss.scalar_type() != at::kFloat) refuse("dloss must be one float32 value");
  const int64_t tokens = l.t.size(0);
  const Tensor& slope = tensor(a[2], "slope");
  if (slope.dim() != 2 || slope.size(0) < 1 || tokens % slope.size(0))
    refuse("slope must be [sequences, experts] with sequences a divisor of the tokens");
  table(a[2], {slope.size(0), l.t.size(1)}, at::kFloat, "slope");
  const int dtype = dtype_of(l.t), score = score_of(a[3]);
  const uint8_t* mask = mask_of(a[4], tokens);
  const uint32_t n = narrow(l.width, "zc_moe_balance_backward");
  const Launch on(a[6], l.t);
  Tensor dlogits = on.output(a[5], l.t.sizes(), l.t.scalar_type(), "dlogits");
  check(without_gil([&] {
          return zc_moe_balance_backward(static_cast<const float*>(dloss.const_data_ptr()), l.p(), dtype, l.stride,
                                         l.rows, n, score, static_cast<uint64_t>(slope.size(0)), mask,
                                         static_cast<const float*>(slope.const_data_ptr()), dlogits.mutable_data_ptr(),
                                         on.stream());
        }),
        "zc_moe_balance_backward");
  return pack({dlogits});
}

// What a dropout draws from.
struct Draw {
  double p;
  const int64_t* rng = nullptr;
  uint32_t call;
  Draw(PyObject* p_, PyObject* rng_, PyObject* call_) : p(PyFloat_AsDouble(p_)) {
    if (p == -1.0 && PyErr_Occurred()) throw Raised();
    if (!(p >= 0.0 && p <= 1.0)) refuse("p must be a probability");
    const long c = integer(call_);
    if (c < 0 || c > 0xFFFFFFFFl) refuse("call must be a number of 32 bits");
    call = static_cast<uint32_t>(c);
    if (rng_ != Py_None) rng = static_cast<const int64_t*>(table(rng_, {2}, at::kLong, "rng").const_data_ptr());
  }
};

// (x, p, rng, call, residual, residual_scale, out, stream) -> (out,)
PyObject* dropout(Args a) {
  const Matrix x = matrix(a[0], "x");
  const int dtype = dtype_of(x.t);
  const Draw draw(a[1], a[2], a[3]);
  if (!draw.rng) refuse("dropout takes a generator's state");
  const void* residual = nullptr;
  uint64_t residual_stride = 0;
  if (a[4] != Py_None) {
    const Matrix r = same_as(a[4], x.t, "residual");
    residual = r.p();
    residual_stride = r.stride;
  }
  const float scale = real(a[5]);
  const uint32_t width = narrow(x.width, "zc_dropout");
  const Launch on(a[7], x.t);
  Tensor out = on.output(a[6], x.t.sizes(), x.t.scalar_type(), "out");
  check(without_gil([&] {
          return zc_dropout(x.p(), dtype, x.stride, residual, residual_stride, scale, x.rows, width, draw.p, draw.rng,
                            draw.call, out.mutable_data_ptr(), on.stream());
        }),
        "zc_dropout");
  return pack({out});
}

// A weight or bias of a layer norm, of the activations' type or float32; NULL for None.
const void* norm_vector(PyObject* o, const Tensor& x, at::ScalarType kind, const char* what) {
  if (o == Py_None) return nullptr;
  const Tensor& t = tensor(o, what);
  if (t.scalar_type() != kind || (kind != x.scalar_type() && kind != at::kFloat))
    refuse("weight and bias must both have the activations' type, or both be float32");
  if (t.dim() != 1 || t.size(0) != x.size(1))
    refuse(std::string(what) + " must have the activations' width, not " + shape_of(t));
  if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
  return t.const_data_ptr();
}

// (y or None, x, weight, bias or None, p, rng, call, residual_scale, eps, x_new, h, save, stream) ->
// (x_new or None, h, stats or None)
PyObject* layer_norm(Args a) {
  zc_layer_norm_args n = {};
  const bool branch = a[0] != Py_None;
  const Matrix x = matrix(a[1], "x");
  if (branch) {
    const Matrix y = same_as(a[0], x.t, "y");
    n.y = y.p();
    n.y_stride = y.stride;
  }
  const Draw draw(a[4], a[5], a[6]);
  if (draw.p > 0 && !draw.rng) refuse("dropout takes a generator's state");
  if (draw.p > 0) n.rng = draw.rng, n.p = draw.p, n.call = draw.call;
  n.x = x.p();
  n.x_stride = x.stride;
  n.tokens = x.rows;
  n.hidden = narrow(x.width, "zc_layer_norm");
  n.dtype = dtype_of(x.t);
  const at::ScalarType kind = tensor(a[2], "weight").scalar_type();
  n.weight = norm_vector(a[2], x.t, kind, "weight");
  n.bias = norm_vector(a[3], x.t, kind, "bias");
  n.params_f32 = kind == at::kFloat && x.t.scalar_type() != at::kFloat;
  n.residual_scale = real(a[7]);
  n.eps = real(a[8]);
  const bool save = truth(a[11]);
  const Launch on(a[12], x.t);
  Tensor x_new, stats;
  if (branch) x_new = on.output(a[9], x.t.sizes(), x.t.scalar_type(), "x_new");
  Tensor h = on.output(a[10], x.t.sizes(), x.t.scalar_type(), branch ? "h" : "out");
  if (save) stats = on.fresh({x.t.size(0), 2}, at::kFloat);
  if (branch) n.x_new = x_new.mutable_data_ptr();
  n.h = h.mutable_data_ptr();
  if (save) n.stats = static_cast<float*>(stats.mutable_data_ptr());
  check(without_gil([&] { return zc_layer_norm(&n, on.stream()); }), "zc_layer_norm");
  return pack({x_new, h, stats});
}

// (dx_new or None, dh, x_new, stats, weight, bias wanted, p, rng, call, residual_scale, branch, ws,
// stream) -> (dy or None, dx, dweight, dbias or None); dy is dx where they are the same
PyObject* layer_norm_backward(Args a) {
  zc_layer_norm_backward_args n = {};
  const Matrix x = matrix(a[2], "x_new"), dh = same_as(a[1], x.t, "dh");
  const bool bias = truth(a[5]), branch = truth(a[10]);
  n.dh = dh.p();
  n.dh_stride = dh.stride;
  n.x_new = x.p();
  n.x_new_stride = x.stride;
  if (a[0] != Py_None) {
    const Matrix m = same_as(a[0], x.t, "dx_new");
    n.dx_new = m.p();
    n.dx_new_stride = m.stride;
  }
  n.stats = static_cast<const float*>(table(a[3], {x.t.size(0), 2}, at::kFloat, "stats").const_data_ptr());
  const Draw draw(a[6], a[7], a[8]);
  if (draw.p > 0 && !draw.rng) refuse("dropout takes a generator's state");
  if (draw.p > 0) n.rng = draw.rng, n.p = draw.p, n.call = draw.call;
  n.tokens = x.rows;
  n.hidden = narrow(x.width, "zc_layer_norm_backward");
  n.dtype = dtype_of(x.t);
  const at::ScalarType kind = tensor(a[4], "weight").scalar_type();
  n.weight = norm_vector(a[4], x.t, kind, "weight");
  if (!n.weight && x.t.size(1)) refuse("the norm takes a weight");
  n.params_f32 = kind == at::kFloat && x.t.scalar_type() != at::kFloat;
  n.residual_scale = real(a[9]);
  if (!branch) n.residual_scale = 1.f;
  const Tensor& ws = tensor(a[11], "ws");
  if (!ws.is_contiguous()) refuse("libzc takes contiguous tensors");
  const Launch on(a[12], x.t);
  Tensor dx = on.fresh(x.t.sizes(), x.t.scalar_type()), dy, dbias;
  if (branch) dy = n.rng || n.residual_scale != 1.f ? on.fresh(x.t.sizes(), x.t.scalar_type()) : dx;
  Tensor dweight = on.fresh({x.t.size(1)}, kind);
  if (bias) dbias = on.fresh({x.t.size(1)}, kind);
  n.dx = dx.mutable_data_ptr();
  if (branch && !dy.is_same(dx)) n.dy = dy.mutable_data_ptr();
  n.dweight = dweight.mutable_data_ptr();
  if (dbias.defined()) n.dbias = dbias.mutable_data_ptr();
  n.ws = ws.mutable_data_ptr();
  n.ws_bytes = static_cast<uint64_t>(ws.nbytes());
  check(without_gil([&] { return zc_layer_norm_backward(&n, on.stream()); }), "zc_layer_norm_backward");
  return pack({dy, dx, dweight, dbias});
}

// Token ids, int32 or int64.
const Tensor& ids_of(PyObject* o) {
  const Tensor& t = tensor(o, "ids");
  if (t.dim() != 1 || (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong))
    refuse("ids must be int32 or int64 [tokens]");
  if (!t.is_contiguous()) refuse("libzc takes contiguous tensors");
  return t;
}

// A torch.dtype, or `otherwise` for None; of two types that go together, the activations' `type` and
// the table's: the same, or float32 for the table.
at::ScalarType kind_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o)) refuse("dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int check_kinds(at::ScalarType rows, at::ScalarType table) {
  if (rows != table && table != at::kFloat) refuse("the table must have the rows' type, or be float32");
  switch (rows) {
    case at::kBFloat16: return ZC_BF16;
    case at::kHalf: return ZC_F16;
    case at::kFloat: return ZC_F32;
    default: refuse("rows are bfloat16, float16 or float32");
  }
}

// (ids, table, status, scale, dtype, out, stream) -> (out,)
PyObject* embedding(Args a) {
  const Tensor& ids = ids_of(a[0]);
  const Matrix t = matrix(a[1], "table");
  const Tensor& status = table(a[2], {1}, at::kInt, "status");
  const float scale = real(a[3]);
  const at::ScalarType kind = kind_of(a[4], t.t.scalar_type());
  const int dtype = check_kinds(kind, t.t.scalar_type());
  const uint32_t hidden = narrow(t.width, "zc_embedding");
  const Launch on(a[6], t.t);
  Tensor out = on.output(a[5], {ids.size(0), t.t.size(1)}, kind, "out");
  check(without_gil([&] {
          return zc_embedding(ids.const_data_ptr(), ids.scalar_type() == at::kLong,
                              static_cast<uint64_t>(ids.size(0)), t.p(), dtype, t.t.scalar_type() == at::kFloat,
                              t.stride, t.rows, hidden, scale, out.mutable_data_ptr(),
                              static_cast<int32_t*>(status.mutable_data_ptr()), on.stream());
        }),
        "zc_embedding");
  return pack({out});
}

// (dout, ids, vocab, ws, status, scale, dtype, dtable or None, accumulate, stream) -> (dtable,)
PyObject* embedding_backward(Args a) {
  const Matrix g = matrix(a[0], "dout");
  const Tensor& ids = ids_of(a[1]);
  if (ids.size(0) != g.t.size(0)) refuse("dout must be [tokens, hidden]");
  const int64_t vocab = integer(a[2]);
  if (vocab < 0) refuse("vocab must not be negative");
  const Tensor& ws = tensor(a[3], "ws");
  if (!ws.is_contiguous()) refuse("libzc takes contiguous tensors");
  const Tensor& status = table(a[4], {1}, at::kInt, "status");
  const float scale = real(a[5]);
  const bool given = a[7] != Py_None, accumulate = truth(a[8]);
  if (accumulate && !given) refuse("accumulate adds to a given dtable");
  at::ScalarType kind = kind_of(a[6], given ? tensor(a[7], "dtable").scalar_type() : g.t.scalar_type());
  const int dtype = check_kinds(g.t.scalar_type(), kind);
  const uint32_t hidden = narrow(g.width, "zc_embedding_backward");
  if (vocab > 0x7FFFFFFF) check(ZC_ERR_TOO_LARGE, "zc_embedding_backward");
  const Launch on(a[9], g.t);
  Tensor dtable = on.output(a[7], {vocab, g.t.size(1)}, kind, "dtable");
  check(without_gil([&] {
          return zc_embedding_backward(g.p(), dtype, g.stride, ids.const_data_ptr(), ids.scalar_type() == at::kLong,
                                       g.rows, static_cast<uint64_t>(vocab), hidden, scale, kind == at::kFloat,
                                       accumulate, dtable.mutable_data_ptr(), ws.mutable_data_ptr(),
                                       static_cast<uint64_t>(ws.nbytes()),
                                       static_cast<int32_t*>(status.mutable_data_ptr()), on.stream());
        }),
        "zc_embedding_backward");
  return pack({dtable});
}

template <PyObject* (*F)(Args), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    // Outputs are new tensors outside autograd: their creation goes straight to the allocation.
    at::AutoDispatchBelowADInplaceOrView plain;
    one_device(args, n);
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(Args), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<moe_route, 9>("moe_route"),
    method<moe_route_backward, 8>("moe_route_backward"),
    method<moe_dispatch, 6>("moe_dispatch"),
    method<moe_combine, 6>("moe_combine"),
    method<moe_combine_backward, 8>("moe_combine_backward"),
    method<norm_forward, 10>("norm_forward"),
    method<norm_backward, 11>("norm_backward"),
    method<moe_balance, 7>("moe_balance"),
    method<moe_balance_backward, 7>("moe_balance_backward"),
    method<dropout, 8>("dropout"),
    method<layer_norm, 13>("layer_norm"),
    method<layer_norm_backward, 13>("layer_norm_backward"),
    method<embedding, 7>("embedding"),
    method<embedding_backward, 10>("embedding_backward"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_zc_torch", "torch entry points of libzc (zc_torch.cpp)", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__zc_torch() { return PyModule_Create(&g_module); }
