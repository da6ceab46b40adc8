// The calls of the expert layer and of a dense layer in 8 bits on torch tensors
// in one step, for the modules experts.py and dense.py: checks, outputs, stream
// and the C call, without a Python statement or a ctypes conversion in between.
// A decode step makes some five of these calls a layer, whose kernels take 2 us
// each where a call through ctypes takes the host 13 to 17 us.
//
// A function returns None for whatever it does not take: a wrong argument, a
// tensor of another device than the current one, a call that the library
// refuses.  The caller then goes the long way, which says what is wrong.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>

#include "ar_rmsnorm.h"

namespace {

// The library's entry points (of the checking build, if that is loaded).
decltype(&ar_route_experts) p_route = nullptr;
decltype(&ar_w4_matvec) p_matvec = nullptr;
decltype(&ar_w4_matvec_experts) p_experts = nullptr;
decltype(&ar_combine) p_combine = nullptr;
decltype(&ar_combine_rmsnorm) p_combine_norm = nullptr;
decltype(&ar_block_rmsnorm) p_block_norm = nullptr;
decltype(&ar_block_rmsnorm_i8) p_block_norm_i8 = nullptr;
decltype(&ar_i8_quantize) p_quantize = nullptr;
decltype(&ar_i8_matmul) p_i8_matmul = nullptr;

struct Unusual {};  // thrown where the long way is to be taken

void want(bool ok) {
  if (!ok) throw Unusual();
}

const at::Tensor &tensor(PyObject *o) {
  want(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// The current device, if that is the tensor's.
int current_device_of(const at::Tensor &t) {
  want(t.is_cuda());
  const int dev = t.get_device();
  want(dev == c10::cuda::current_device());
  return dev;
}

bool is_like(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.is_contiguous() &&
         t.sizes() == shape;
}

const void *input(PyObject *o, at::ScalarType type, at::IntArrayRef shape, int dev) {
  const at::Tensor &t = tensor(o);
  want(is_like(t, type, shape, dev));
  return t.const_data_ptr();
}
const void *optional(PyObject *o, at::ScalarType type, at::IntArrayRef shape, int dev) {
  return o == Py_None ? nullptr : input(o, type, shape, dev);
}

// An output: the caller's tensor, or a new one (straight from the caching
// allocator: through the dispatcher each takes 0.5 us more).
struct Output {
  at::Tensor t;
  void *p;
  Output(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const at::Tensor &like, int dev) {
    if (o == Py_None) {
      t = at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
    } else {
      t = tensor(o);
      want(is_like(t, type, shape, dev));
    }
    p = t.mutable_data_ptr();
  }
};

int type_code(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return AR_TYPE_F32;
    case at::kBFloat16: return AR_TYPE_BF16;
    case at::kHalf: return AR_TYPE_F16;
    default: throw Unusual();
  }
}

int whole(PyObject *o) {
  want(PyLong_Check(o));
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  want(over == 0 && v >= INT_MIN && v <= INT_MAX);
  return static_cast<int>(v);
}
float number(PyObject *o) {
  want(PyFloat_Check(o) || PyLong_Check(o));
  const double v = PyFloat_AsDouble(o);
  want(!PyErr_Occurred());
  return static_cast<float>(v);
}

// Makes the call without the interpreter's lock.
template <typename F>
void call(int dev, F f) {
  void *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  int st;
  Py_BEGIN_ALLOW_THREADS;
  st = f(stream);
  Py_END_ALLOW_THREADS;
  want(st == AR_OK);
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b) {
  PyObject *x = THPVariable_Wrap(a), *y = x ? THPVariable_Wrap(b) : nullptr;
  PyObject *both = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
}

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t wanted, F f) {
  if (n != wanted) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", wanted, n);
    return nullptr;
  }
  try {
    return f();
  } catch (...) {  // the long way finds the reason again
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// (logits, k, bias, scoring, groups, topk_groups, group_score, renorm, scale,
// weights, ids) -> (weights, ids)
PyObject *route_experts(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const at::Tensor &logits = tensor(v[0]);
    const int dev = current_device_of(logits);
    const int type = type_code(logits);
    want(logits.dim() == 2);
    const int64_t m = logits.size(0), E = logits.size(1);
    want((logits.stride(1) == 1 || E <= 1) && E <= INT_MAX);
    const int64_t row = m <= 1 ? E : logits.stride(0);
    const int k = whole(v[1]);
    want(k > 0);
    const void *bias = optional(v[2], at::kFloat, {E}, dev);
    const int scoring = whole(v[3]), groups = whole(v[4]);
    const int topk_groups = v[5] == Py_None ? groups : whole(v[5]);
    const int group_score = whole(v[6]);
    const int renorm = PyObject_IsTrue(v[7]);
    want(renorm >= 0);
    const float scale = number(v[8]);
    Output w(v[9], at::kFloat, {m, k}, logits, dev), ids(v[10], at::kInt, {m, k}, logits, dev);
    const void *x = logits.const_data_ptr();
    call(dev, [&](void *stream) {
      return p_route(x, type, row, static_cast<const float *>(bias), m, static_cast<int>(E), k,
                     scoring, groups, topk_groups, group_score, renorm, scale,
                     static_cast<float *>(w.p), static_cast<int32_t *>(ids.p), stream);
    });
    return pair(w.t, ids.t);
  });
}

// 4-bit weights [*lead, N, K / 2] and what goes with them.
struct Weights {
  const void *q, *scales, *zeros;
  int type, group;
  int64_t N;
  Weights(PyObject *q_, PyObject *scales_, PyObject *zeros_, int64_t K, int lead, int dev) {
    const at::Tensor &tq = tensor(q_), &ts = tensor(scales_);
    want(tq.dim() == lead + 2 && ts.dim() == lead + 2);
    const int64_t ng = ts.size(lead + 1);
    want(ng >= 1 && K > 0 && K % ng == 0 && K / ng <= INT_MAX && tq.size(lead + 1) * 2 == K);
    int64_t shape[3] = {tq.size(0), tq.size(lead), ng};
    if (lead == 0) shape[1] = ng;
    const at::IntArrayRef of_s(shape, lead + 2);
    type = type_code(ts);
    q = input(q_, at::kByte, tq.sizes(), dev);
    scales = input(scales_, ts.scalar_type(), of_s, dev);
    zeros = optional(zeros_, at::kByte, of_s, dev);
    group = static_cast<int>(K / ng);
    N = tq.size(lead);
  }
};

// (x, q, scales, zeros, act, out) -> out
PyObject *w4_matvec(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    const at::Tensor &tx = tensor(v[0]);
    const int dev = current_device_of(tx);
    want(tx.dim() == 2);
    const int64_t m = tx.size(0), K = tx.size(1);
    const void *x = input(v[0], at::kBFloat16, tx.sizes(), dev);
    const Weights w(v[1], v[2], v[3], K, 0, dev);
    const int act = whole(v[4]);
    Output out(v[5], at::kBFloat16, {m, act == AR_ACT_SILU_MUL ? w.N / 2 : w.N}, tx, dev);
    call(dev, [&](void *stream) {
      return p_matvec(x, w.q, w.scales, w.type, w.zeros, m, w.N, K, w.group, act, out.p, stream);
    });
    return THPVariable_Wrap(out.t);
  });
}

// (x, ids, q, scales, zeros, act, first, out) -> out
PyObject *w4_matvec_experts(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    const at::Tensor &tx = tensor(v[0]), &ti = tensor(v[1]);
    const int dev = current_device_of(tx);
    want(ti.dim() == 2 && (tx.dim() == 2 || tx.dim() == 3));
    const int64_t m = ti.size(0), k = ti.size(1), K = tx.size(-1);
    const bool per_pair = tx.dim() == 3;
    want(k <= INT_MAX);
    const int64_t shape[3] = {m, per_pair ? k : K, K};
    const void *x = input(v[0], at::kBFloat16, at::IntArrayRef(shape, per_pair ? 3 : 2), dev);
    const void *ids = input(v[1], at::kInt, ti.sizes(), dev);
    const Weights w(v[2], v[3], v[4], K, 1, dev);
    const int64_t E = THPVariable_Unpack(v[2]).size(0);
    want(E <= INT_MAX);
    const int act = whole(v[5]), first = whole(v[6]);
    Output out(v[7], at::kBFloat16, {m, k, act == AR_ACT_SILU_MUL ? w.N / 2 : w.N}, tx, dev);
    call(dev, [&](void *stream) {
      return p_experts(x, per_pair ? 1 : 0, static_cast<const int32_t *>(ids), m,
                       static_cast<int>(k), w.q, w.scales, w.type, w.zeros, first,
                       static_cast<int>(E), w.N, K, w.group, act, out.p, stream);
    });
    return THPVariable_Wrap(out.t);
  });
}

// What the two combine calls share: (y, weights, shared, slots).
struct Summands {
  int dev, k;
  int64_t m, H, rows;
  const void *y, *weights, *shared, *slots;
  Summands(PyObject *y_, PyObject *weights_, PyObject *shared_, PyObject *slots_) {
    const at::Tensor &ty = tensor(y_), &tw = tensor(weights_);
    dev = current_device_of(ty);
    want(tw.dim() == 2 && tw.size(1) <= INT_MAX);
    m = tw.size(0);
    k = static_cast<int>(tw.size(1));
    weights = input(weights_, at::kFloat, tw.sizes(), dev);
    const bool slotted = slots_ != Py_None;
    want(ty.dim() == (slotted ? 2 : 3));
    H = ty.size(-1);
    rows = slotted ? ty.size(0) : m * k;
    y = slotted ? input(y_, at::kBFloat16, {rows, H}, dev) : input(y_, at::kBFloat16, {m, k, H}, dev);
    slots = optional(slots_, at::kInt, tw.sizes(), dev);
    shared = optional(shared_, at::kBFloat16, {m, H}, dev);
  }
};

// (y, weights, shared, slots, out) -> out
PyObject *combine(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject * {
    const Summands s(v[0], v[1], v[2], v[3]);
    Output out(v[4], at::kBFloat16, {s.m, s.H}, THPVariable_Unpack(v[0]), s.dev);
    call(s.dev, [&](void *stream) {
      return p_combine(s.y, s.rows, static_cast<const int32_t *>(s.slots),
                       static_cast<const float *>(s.weights), s.shared, s.m, s.k, s.H, out.p, stream);
    });
    return THPVariable_Wrap(out.t);
  });
}

// (y, weights, residual, weight, eps, shared, slots, out, residual_out) ->
// (out, residual_out)
PyObject *combine_rmsnorm(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const Summands s(v[0], v[1], v[5], v[6]);
    const void *residual = input(v[2], at::kBFloat16, {s.m, s.H}, s.dev);
    const void *weight = input(v[3], at::kBFloat16, {s.H}, s.dev);
    const float eps = number(v[4]);
    const at::Tensor &like = THPVariable_Unpack(v[0]);
    Output out(v[7], at::kBFloat16, {s.m, s.H}, like, s.dev);
    Output rout(v[8], at::kBFloat16, {s.m, s.H}, like, s.dev);
    call(s.dev, [&](void *stream) {
      return p_combine_norm(s.y, s.rows, static_cast<const int32_t *>(s.slots),
                            static_cast<const float *>(s.weights), s.shared, residual, weight, eps,
                            s.m, s.k, s.H, out.p, rout.p, stream);
    });
    return pair(out.t, rout.t);
  });
}

int type16_code(const at::Tensor &t) {
  want(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf);
  return type_code(t);
}

// (partials, residual, weight, eps, post_weight, gate, block_scale,
// residual_scale, weight_offset, bytes, out or q, scales, residual_out) ->
// (out, residual_out) or (q, scales, residual_out)
PyObject *block_rmsnorm(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject * {
    want(PyList_Check(v[0]) || PyTuple_Check(v[0]));
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(v[0]);
    want(count >= 1 && count <= AR_MAX_RANKS);
    PyObject **items = PySequence_Fast_ITEMS(v[0]);
    const at::Tensor &first = tensor(items[0]);
    const int dev = current_device_of(first);
    const int type = type16_code(first);
    const at::ScalarType dtype = first.scalar_type();
    want(first.dim() == 2);
    const int64_t m = first.size(0), H = first.size(1);
    const void *partials[AR_MAX_RANKS];
    for (Py_ssize_t k = 0; k < count; ++k) partials[k] = input(items[k], dtype, {m, H}, dev);
    const at::ScalarType rdtype = tensor(v[1]).scalar_type();
    want(rdtype == dtype || rdtype == at::kFloat);
    const void *residual = input(v[1], rdtype, {m, H}, dev);
    const void *weight = input(v[2], dtype, {H}, dev), *post = optional(v[4], dtype, {H}, dev);
    const float eps = number(v[3]);
    const void *gate = nullptr;
    int64_t gate_stride = H, gate_rows = 1;
    if (v[5] != Py_None) {
      const at::Tensor &t = tensor(v[5]);
      want(t.scalar_type() == dtype && t.is_cuda() && t.get_device() == dev);
      want((t.dim() == 1 || t.dim() == 2) && t.size(-1) == H && (t.stride(-1) == 1 || H <= 1));
      const int64_t g = t.dim() == 2 ? t.size(0) : 1;
      want(g >= 1 && m >= 1 && m % g == 0);
      if (g > 1) gate_stride = t.stride(0);
      gate_rows = m / g;
      gate = t.const_data_ptr();
    }
    const float block_scale = number(v[6]), residual_scale = number(v[7]), offset = number(v[8]);
    const bool bytes = v[9] == Py_True;
    Output out(v[10], bytes ? at::kChar : dtype, {m, H}, first, dev);
    Output rout(v[12], rdtype, {m, H}, first, dev);
    const int rtype = rdtype == at::kFloat ? AR_TYPE_F32 : type, parts = static_cast<int>(count);
    if (!bytes) {
      call(dev, [&](void *stream) {
        return p_block_norm(partials, parts, type, post, gate, gate_stride, gate_rows, block_scale,
                            residual, rtype, residual_scale, weight, offset, eps, m, H, out.p, rout.p,
                            stream);
      });
      return pair(out.t, rout.t);
    }
    Output scales(v[11], at::kFloat, {m}, first, dev);
    call(dev, [&](void *stream) {
      return p_block_norm_i8(partials, parts, type, post, gate, gate_stride, gate_rows, block_scale,
                             residual, rtype, residual_scale, weight, offset, eps, m, H,
                             static_cast<int8_t *>(out.p), static_cast<float *>(scales.p), rout.p,
                             stream);
    });
    PyObject *a = THPVariable_Wrap(out.t), *b = a ? THPVariable_Wrap(scales.t) : nullptr;
    PyObject *c = b ? THPVariable_Wrap(rout.t) : nullptr;
    PyObject *all = c ? PyTuple_Pack(3, a, b, c) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    Py_XDECREF(c);
    return all;
  });
}

// (x, q, scales) -> (q, scales)
PyObject *i8_quantize(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject * {
    const at::Tensor &x = tensor(v[0]);
    const int dev = current_device_of(x);
    const int type = type16_code(x);
    want(x.dim() == 2);
    const int64_t m = x.size(0), K = x.size(1);
    want(x.stride(1) == 1 || K <= 1);
    const int64_t row = m <= 1 ? K : x.stride(0);
    Output q(v[1], at::kChar, {m, K}, x, dev), scales(v[2], at::kFloat, {m}, x, dev);
    const void *from = x.const_data_ptr();
    call(dev, [&](void *stream) {
      return p_quantize(from, type, row, m, K, static_cast<int8_t *>(q.p),
                        static_cast<float *>(scales.p), stream);
    });
    return pair(q.t, scales.t);
  });
}

// (x, x_scales, w, w_scales, act, type, out) -> out
PyObject *i8_matmul(PyObject *, PyObject *const *v, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    const at::Tensor &tx = tensor(v[0]), &tw = tensor(v[2]);
    const int dev = current_device_of(tx);
    want(tx.dim() == 2 && tw.dim() == 2);
    const int64_t m = tx.size(0), K = tx.size(1), N = tw.size(0);
    const void *x = input(v[0], at::kChar, {m, K}, dev), *xs = input(v[1], at::kFloat, {m}, dev);
    const void *w = input(v[2], at::kChar, {N, K}, dev), *ws = input(v[3], at::kFloat, {N}, dev);
    const int act = whole(v[4]), type = whole(v[5]);
    const at::ScalarType dtype = type == AR_TYPE_F32    ? at::kFloat
                                 : type == AR_TYPE_BF16 ? at::kBFloat16
                                                        : at::kHalf;
    Output out(v[6], dtype, {m, act == AR_ACT_SILU_MUL ? N / 2 : N}, tx, dev);
    call(dev, [&](void *stream) {
      return p_i8_matmul(static_cast<const int8_t *>(x), static_cast<const float *>(xs),
                         static_cast<const int8_t *>(w), static_cast<const float *>(ws), m, N, K, act,
                         type, out.p, stream);
    });
    return THPVariable_Wrap(out.t);
  });
}

template <typename F>
void take(F *&to, void *from) {
  static_assert(sizeof(to) == sizeof(from), "one address");
  std::memcpy(&to, &from, sizeof(from));
}

// Takes the addresses of the library's entry points, in the order above.
PyObject *bind(PyObject *, PyObject *const *v, Py_ssize_t n) {
  constexpr int kCalls = 9;
  void *at[kCalls];
  if (n != kCalls) {
    PyErr_SetString(PyExc_TypeError, "nine addresses");
    return nullptr;
  }
  for (int i = 0; i < kCalls; ++i) {
    at[i] = PyLong_AsVoidPtr(v[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  take(p_route, at[0]);
  take(p_matvec, at[1]);
  take(p_experts, at[2]);
  take(p_combine, at[3]);
  take(p_combine_norm, at[4]);
  take(p_block_norm, at[5]);
  take(p_block_norm_i8, at[6]);
  take(p_quantize, at[7]);
  take(p_i8_matmul, at[8]);
  Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL,
          nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<route_experts>("route_experts"),
                         method<w4_matvec>("w4_matvec"),
                         method<w4_matvec_experts>("w4_matvec_experts"),
                         method<combine>("combine"),
                         method<combine_rmsnorm>("combine_rmsnorm"),
                         method<block_rmsnorm>("block_rmsnorm"),
                         method<i8_quantize>("i8_quantize"),
                         method<i8_matmul>("i8_matmul"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
