// The torch-facing calls of the operators at the block's edge (moe.route, moe.norm_forward, ...)
// without the interpreter's share: argument checks, outputs from torch's allocator, the current
// stream and the C ABI call in one step.  A small batch's pass costs the host more than the GPU
// (a routed token 10.2 us through ctypes, 5.5 here; a norm 12.8 and 6.7).  Each function handles the plain call (dense
// CUDA tensors of one device, the current one, outputs not given) and returns None for any other,
// and for every error, which the Python wrapper then takes the long way and names.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxfp4_moe.h"

namespace {

struct Entry {  // the loaded library's entry points (release or debug build)
  decltype(&mxfp4_moe_route) route;
  decltype(&mxfp4_moe_route_backward) route_backward;
  decltype(&mxfp4_moe_norm_forward) norm_forward;
  decltype(&mxfp4_moe_norm_workspace_size) norm_workspace_size;
  decltype(&mxfp4_moe_norm_backward) norm_backward;
  decltype(&mxfp4_moe_checkpoint_pack) checkpoint_pack;
  decltype(&mxfp4_moe_checkpoint_unpack) checkpoint_unpack;
} entry;

// The call is not a plain one.
struct Other {};

bool given(PyObject* o) { return o != Py_None; }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Other{};
  return THPVariable_Unpack(o);
}

// A dense tensor with elements and memory, of that type and shape, on `device`.
const at::Tensor& dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor& t = tensor(o);
  if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device ||
      t.scalar_type() != type || t.sizes() != shape || t.numel() == 0 || !t.is_contiguous() ||
      !t.data_ptr())
    throw Other{};
  return t;
}

int current_device_of(const at::Tensor& t) {
  if (!t.is_cuda() || t.dim() != 2 || t.get_device() != c10::cuda::current_device()) throw Other{};
  if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX) throw Other{};
  return (int)t.get_device();
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}

PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

template <class... T>
PyObject* tuple_of(const T&... t) {
  PyObject* out = PyTuple_New(sizeof...(t));
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(out, i++, wrap(t)), ...);
  return out;
}

int number(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if ((v == -1 && PyErr_Occurred()) || v != (int)v) throw Other{};
  return (int)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Other{};
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Other{};
  return v != 0;
}
int named(PyObject* o, const char* zero, const char* one) {
  if (!PyUnicode_Check(o)) throw Other{};
  if (PyUnicode_CompareWithASCIIString(o, zero) == 0) return 0;
  if (PyUnicode_CompareWithASCIIString(o, one) == 0) return 1;
  throw Other{};
}
int scores_of(PyObject* o) { return named(o, "softmax", "sigmoid"); }
int kind_of(PyObject* o) { return named(o, "layer", "rms"); }
int format_of(PyObject* o) { return named(o, "e4m3", "int8"); }
int rows_format_of(at::ScalarType t) {
  if (t == at::kBFloat16) return MXFP4_MOE_ROWS_BF16;
  if (t == at::kFloat) return MXFP4_MOE_ROWS_FP32;
  throw Other{};
}
void done(int rc) {
  if (rc != MXFP4_MOE_OK) throw Other{};
}

// Runs one call; whatever keeps it from being a plain one is None.
template <class F>
PyObject* plain(Py_ssize_t n, Py_ssize_t want, const F& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// k, scores, groups, top_groups, group_best, renormalize, scale
mxfp4_moe_routing routing_of(PyObject* const* a, const at::Tensor& logits) {
  return {(int32_t)logits.size(0), (int32_t)logits.size(1), number(a[0]), scores_of(a[1]),
          number(a[2]), number(a[3]), number(a[4]), truth(a[5]), real(a[6])};
}

// (routing x 7, logits, bias) -> (topk_idx, topk_w)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 9, [&]() -> PyObject* {
    const at::Tensor& logits = tensor(a[7]);
    const int dev = current_device_of(logits);
    const mxfp4_moe_routing r = routing_of(a, logits);
    if (r.k < 1) throw Other{};
    dense(a[7], at::kFloat, {r.T, r.E}, dev);
    const float* bias = given(a[8]) ? (const float*)dense(a[8], at::kFloat, {r.E}, dev).data_ptr() : nullptr;
    const at::Tensor idx = fresh({r.T, r.k}, at::kInt, dev), w = fresh({r.T, r.k}, at::kFloat, dev);
    done(entry.route(&r, (const float*)logits.data_ptr(), bias, (int32_t*)idx.data_ptr(),
                     (float*)w.data_ptr(), nullptr, stream_of(dev)));
    return tuple_of(idx, w);
  });
}

// (routing x 7, logits, topk_idx, topk_w, d_topk_w) -> d_logits
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 11, [&]() -> PyObject* {
    const at::Tensor& logits = tensor(a[7]);
    const int dev = current_device_of(logits);
    const mxfp4_moe_routing r = routing_of(a, logits);
    dense(a[7], at::kFloat, {r.T, r.E}, dev);
    const at::Tensor &idx = dense(a[8], at::kInt, {r.T, r.k}, dev),
                     &w = dense(a[9], at::kFloat, {r.T, r.k}, dev),
                     &dw = dense(a[10], at::kFloat, {r.T, r.k}, dev);
    const at::Tensor d = fresh({r.T, r.E}, at::kFloat, dev);
    done(entry.route_backward(&r, (const float*)logits.data_ptr(), (const int32_t*)idx.data_ptr(),
                              (const float*)w.data_ptr(), (const float*)dw.data_ptr(),
                              (float*)d.data_ptr(), stream_of(dev)));
    return wrap(d);
  });
}

// Rows, or the codes, scales and format of a checkpoint (codes None: rows).
struct Rows {
  int T, H, dev;
  const at::Tensor* t;
  const void* x = nullptr;
  mxfp4_moe_checkpoint from{};
  const mxfp4_moe_checkpoint* checkpoint() const { return x ? nullptr : &from; }
  Rows(PyObject* rows, PyObject* scales, PyObject* format) : t(&tensor(rows)) {
    dev = current_device_of(*t);
    T = (int)t->size(0);
    H = (int)t->size(1);
    if (!given(scales)) {
      x = dense(rows, t->scalar_type(), {T, H}, dev).data_ptr();
    } else {
      dense(rows, at::kByte, {T, H}, dev);
      const at::Tensor& s = dense(scales, at::kByte, {T, H / 32}, dev);
      from = {(uint8_t*)t->data_ptr(), (uint8_t*)s.data_ptr(), format_of(format)};
    }
  }
};

const void* vector_of(PyObject* o, int H, int dev, int* format, bool first) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o);
  const int f = rows_format_of(t.scalar_type());
  if (!first && *format != f) throw Other{};
  *format = f;
  return dense(o, t.scalar_type(), {H}, dev).data_ptr();
}

// (rows, scales, format, fp32, y, weight, bias, kind, eps, checkpoint)
//   -> (out, x_out, mean, rstd, codes, scales)
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 10, [&]() -> PyObject* {
    const Rows r(a[0], a[1], a[2]);
    const at::ScalarType type = r.x ? r.t->scalar_type() : truth(a[3]) ? at::kFloat : at::kBFloat16;
    mxfp4_moe_norm d{r.T, r.H, kind_of(a[7]), real(a[8]), rows_format_of(type), 0};
    const void* weight = vector_of(a[5], r.H, r.dev, &d.param_format, true);
    const void* bias = vector_of(a[6], r.H, r.dev, &d.param_format, weight == nullptr);
    at::Tensor x_out, mean, codes, scales;
    const void* y = nullptr;
    if (given(a[4])) {
      y = dense(a[4], type, {r.T, r.H}, r.dev).data_ptr();
      x_out = fresh({r.T, r.H}, type, r.dev);
    }
    mxfp4_moe_checkpoint to{};
    if (given(a[9])) {
      if (r.H % 32) throw Other{};
      codes = fresh({r.T, r.H}, at::kByte, r.dev);
      scales = fresh({r.T, r.H / 32}, at::kByte, r.dev);
      to = {(uint8_t*)codes.data_ptr(), (uint8_t*)scales.data_ptr(), format_of(a[9])};
    }
    const at::Tensor out = fresh({r.T, r.H}, type, r.dev), rstd = fresh({r.T}, at::kFloat, r.dev);
    if (d.kind == MXFP4_MOE_NORM_LAYER) mean = fresh({r.T}, at::kFloat, r.dev);
    done(entry.norm_forward(&d, r.x, r.checkpoint(), y, weight, bias, y ? x_out.data_ptr() : nullptr,
                            to.codes ? &to : nullptr, out.data_ptr(),
                            mean.defined() ? (float*)mean.data_ptr() : nullptr,
                            (float*)rstd.data_ptr(), stream_of(r.dev)));
    return tuple_of(out, x_out, mean, rstd, codes, scales);
  });
}

// (d_out, rows, scales, format, mean, rstd, weight, kind, g) -> (dx, d_weight, d_bias)
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 9, [&]() -> PyObject* {
    const Rows r(a[1], a[2], a[3]);
    const at::Tensor& d_out = tensor(a[0]);
    const at::ScalarType type = d_out.scalar_type();
    if (r.x && r.t->scalar_type() != type) throw Other{};
    dense(a[0], type, {r.T, r.H}, r.dev);
    mxfp4_moe_norm d{r.T, r.H, kind_of(a[7]), 0.f, rows_format_of(type), 0};
    const void* weight = vector_of(a[6], r.H, r.dev, &d.param_format, true);
    const bool layer = d.kind == MXFP4_MOE_NORM_LAYER;
    const void* mean = given(a[4]) ? dense(a[4], at::kFloat, {r.T}, r.dev).data_ptr() : nullptr;
    if (layer && !mean) throw Other{};
    const void* rstd = dense(a[5], at::kFloat, {r.T}, r.dev).data_ptr();
    const void* g = given(a[8]) ? dense(a[8], type, {r.T, r.H}, r.dev).data_ptr() : nullptr;
    size_t bytes = 0;
    done(entry.norm_workspace_size(&d, &bytes));
    const at::Tensor dx = fresh({r.T, r.H}, type, r.dev), dw = fresh({r.H}, at::kFloat, r.dev);
    const at::Tensor db = layer ? fresh({r.H}, at::kFloat, r.dev) : at::Tensor();
    const at::Tensor ws = fresh({(int64_t)bytes}, at::kByte, r.dev);
    done(entry.norm_backward(&d, d_out.data_ptr(), r.x, r.checkpoint(), (const float*)mean,
                             (const float*)rstd, weight, g, dx.data_ptr(), (float*)dw.data_ptr(),
                             layer ? (float*)db.data_ptr() : nullptr, ws.data_ptr(), bytes,
                             stream_of(r.dev)));
    return tuple_of(dx, dw, db);
  });
}

// (rows, format) -> (codes, scales)
PyObject* checkpoint_pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 2, [&]() -> PyObject* {
    const Rows r(a[0], Py_None, Py_None);
    if (r.H % 32) throw Other{};
    const int fmt = rows_format_of(r.t->scalar_type());
    const at::Tensor codes = fresh({r.T, r.H}, at::kByte, r.dev), scales = fresh({r.T, r.H / 32}, at::kByte, r.dev);
    const mxfp4_moe_checkpoint to{(uint8_t*)codes.data_ptr(), (uint8_t*)scales.data_ptr(), format_of(a[1])};
    done(entry.checkpoint_pack(r.T, r.H, fmt, r.x, &to, stream_of(r.dev)));
    return tuple_of(codes, scales);
  });
}

// (codes, scales, format, fp32) -> rows
PyObject* checkpoint_unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plain(n, 4, [&]() -> PyObject* {
    if (!given(a[1])) throw Other{};
    const Rows r(a[0], a[1], a[2]);
    const bool f32 = truth(a[3]);
    const at::Tensor out = fresh({r.T, r.H}, f32 ? at::kFloat : at::kBFloat16, r.dev);
    done(entry.checkpoint_unpack(r.T, r.H, f32 ? MXFP4_MOE_ROWS_FP32 : MXFP4_MOE_ROWS_BF16, &r.from,
                                 out.data_ptr(), stream_of(r.dev)));
    return wrap(out);
  });
}

// The addresses of the loaded library's entry points, in the order of Entry.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5, p + 6)) return nullptr;
  entry = {reinterpret_cast<decltype(entry.route)>(p[0]),
           reinterpret_cast<decltype(entry.route_backward)>(p[1]),
           reinterpret_cast<decltype(entry.norm_forward)>(p[2]),
           reinterpret_cast<decltype(entry.norm_workspace_size)>(p[3]),
           reinterpret_cast<decltype(entry.norm_backward)>(p[4]),
           reinterpret_cast<decltype(entry.checkpoint_pack)>(p[5]),
           reinterpret_cast<decltype(entry.checkpoint_unpack)>(p[6])};
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"route", fast(route), METH_FASTCALL, nullptr},
    {"route_backward", fast(route_backward), METH_FASTCALL, nullptr},
    {"norm_forward", fast(norm_forward), METH_FASTCALL, nullptr},
    {"norm_backward", fast(norm_backward), METH_FASTCALL, nullptr},
    {"checkpoint_pack", fast(checkpoint_pack), METH_FASTCALL, nullptr},
    {"checkpoint_unpack", fast(checkpoint_unpack), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_edge", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__edge(void) { return PyModule_Create(&module); }
