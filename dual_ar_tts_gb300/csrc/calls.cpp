// The 8-bit operators' calls from Python on torch tensors: checks, outputs, launch.  The calls themselves are those of
// include/s2frame.h; this is what a Python function would do around them, in C++, because these calls are short: on a Grace
// core quantize_q8 of one row takes 4.6 us here, 2.1 where its outputs are given (13 through Python and ctypes).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "../../include/s2frame.h"

namespace {

PyObject* s2_error = nullptr;  // the package's S2Error(function, code, message)

struct Bad {
  const char* what;
};
[[noreturn]] void bad(const char* what) { throw Bad{what}; }
constexpr const char* kDevice = "tensors must be on one CUDA device, the operand fp32, bf16 or fp16";

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) bad("a tensor was expected");
  return THPVariable_Unpack(o);
}
const at::Tensor* given(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

int kind(at::ScalarType t) {
  return t == at::kFloat ? S2_F32 : t == at::kBFloat16 ? S2_BF16 : t == at::kHalf ? S2_F16 : -1;
}
int cuda_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }
int whole(int64_t v) { return static_cast<int>(std::min<int64_t>(v, INT_MAX)); }  // the library refuses what is too large
uintptr_t place(const at::Tensor& t) { return reinterpret_cast<uintptr_t>(t.data_ptr()); }

// x [n][k] as rows of neighbouring elements (a copy where they are not), and their stride
struct Rows {
  at::Tensor x;
  int64_t stride;
  explicit Rows(const at::Tensor& t) {
    const int64_t n = t.size(0), k = t.size(1), s0 = n == 1 ? k : t.stride(0);  // of a single row it may be anything
    const bool fine = (t.stride(1) == 1 || k == 1) && s0 >= k;
    x = fine ? t : t.contiguous();
    stride = fine ? s0 : k;
  }
};

// Runs a call on the current stream of the tensors' device, with that device current meanwhile.
template <typename F>
void launch(const char* name, int dev, F call) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const int rc = call(reinterpret_cast<CUstream_st*>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()));
  if (rc == S2_OK) return;
  PyObject* e = PyObject_CallFunction(s2_error, "sis", name, rc, "see include/s2frame.h for what the call takes");
  if (e) {
    PyErr_SetObject(s2_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

// An output: the caller's, or a new one
struct Out {
  at::Tensor t;
  PyObject* o = nullptr;  // the caller's object
  PyObject* object() const {
    if (!o) return THPVariable_Wrap(t);
    Py_INCREF(o);
    return o;
  }
};
Out output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like, const char* what, int align = 1) {
  Out r;
  if (const at::Tensor* g = given(o)) {
    if (g->scalar_type() != type || g->sizes() != shape || cuda_of(*g) != cuda_of(like) || !g->is_contiguous() ||
        place(*g) % align)
      bad(what);
    r.t = *g;
    r.o = o;
  } else {
    r.t = at::empty(shape, like.options().dtype(type).requires_grad(false));
  }
  return r;
}

// codes and scales of a row quantiser
struct Coded {
  Out codes, scales;
  Coded(PyObject* c, PyObject* s, const at::Tensor& x, int64_t cols) {
    codes = output(c, {x.size(0), (cols + 15) / 16 * 16}, at::kChar, x,
                   "codes must be contiguous int8 [rows][columns rounded up to 16] on the operand's device, from 16 bytes on", 16);
    scales = output(s, {x.size(0)}, at::kFloat, x, "scales must be contiguous fp32 [rows] on the operand's device");
  }
  int8_t* code() const { return static_cast<int8_t*>(codes.t.data_ptr()); }
  float* scale() const { return static_cast<float*>(scales.t.data_ptr()); }
  PyObject* pair() const { return tuple(codes.object(), scales.object(), nullptr, 2); }
  static PyObject* tuple(PyObject* a, PyObject* b, PyObject* c, int n) {
    PyObject* t = PyTuple_New(n);
    if (!t || !a || !b || (n == 3 && !c)) {
      Py_XDECREF(t), Py_XDECREF(a), Py_XDECREF(b), Py_XDECREF(c);
      throw python_error();
    }
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    if (n == 3) PyTuple_SET_ITEM(t, 2, c);
    return t;
  }
};

// A row operand's device; checks its type and shape.
int operand(const at::Tensor& x, const char* what) {
  const int dev = cuda_of(x);
  if (dev < 0 || kind(x.scalar_type()) < 0) bad(kDevice);
  if (x.dim() != 2 || x.size(1) < 1) bad(what);
  return dev;
}

PyObject* quantize(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const int dev = operand(x, "quantize_q8 takes [rows][cols]");
  const int64_t n = x.size(0), cols = x.size(1);
  const Coded out(a[1], a[2], x, cols);
  if (n) {
    const Rows r(x);
    launch("s2_quantize_q8", dev, [&](CUstream_st* st) {
      return s2_quantize_q8(r.x.data_ptr(), kind(x.scalar_type()), r.stride, n, whole(cols), out.code(), out.scale(), st);
    });
  }
  return out.pair();
}

PyObject* swiglu(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0]);
  const int dev = operand(x, "swiglu_q8 takes [rows][2 f]");
  if (x.size(1) % 2) bad("swiglu_q8 takes [rows][2 f]");
  const int64_t n = x.size(0), cols = x.size(1) / 2;
  const Coded out(a[1], a[2], x, cols);
  if (n) {
    const Rows r(x);
    launch("s2_swiglu_q8", dev, [&](CUstream_st* st) {
      return s2_swiglu_q8(r.x.data_ptr(), kind(x.scalar_type()), r.stride, n, whole(cols), out.code(), out.scale(), st);
    });
  }
  return out.pair();
}

PyObject* norm(PyObject* const* a) {  // x, weight, eps, residual, total, codes, scales
  const at::Tensor &x = tensor(a[0]), &weight = tensor(a[1]);
  const int dev = operand(x, "rms_norm_q8 takes [rows][cols]");
  const int64_t n = x.size(0), cols = x.size(1);
  const double eps = PyFloat_AsDouble(a[2]);
  if (eps == -1.0 && PyErr_Occurred()) throw python_error();
  if (cuda_of(weight) != dev) bad(kDevice);
  if (weight.scalar_type() != at::kFloat || weight.dim() != 1 || weight.size(0) != cols || !weight.is_contiguous())
    bad("weight must be contiguous fp32 [cols]");
  const at::Tensor* residual = given(a[3]);
  Out total;
  if (residual) {
    if (residual->scalar_type() != x.scalar_type() || residual->sizes() != x.sizes() || cuda_of(*residual) != dev)
      bad("residual must have x's shape and type, on its device");
    total = output(a[4], x.sizes(), x.scalar_type(), x, "total must be contiguous, of x's shape and type, on its device");
  } else if (a[4] != Py_None) {
    bad("total goes with a residual");
  }
  const Coded out(a[5], a[6], x, cols);
  if (n) {
    const Rows r(x);
    if (residual) {
      const Rows s(*residual);
      launch("s2_rms_norm_q8", dev, [&](CUstream_st* st) {
        return s2_rms_norm_q8(r.x.data_ptr(), kind(x.scalar_type()), r.stride, s.x.data_ptr(), s.stride,
                              static_cast<const float*>(weight.data_ptr()), static_cast<float>(eps), n, whole(cols),
                              total.t.data_ptr(), out.code(), out.scale(), st);
      });
    } else {
      launch("s2_rms_norm_q8", dev, [&](CUstream_st* st) {
        return s2_rms_norm_q8(r.x.data_ptr(), kind(x.scalar_type()), r.stride, nullptr, 0,
                              static_cast<const float*>(weight.data_ptr()), static_cast<float>(eps), n, whole(cols), nullptr,
                              out.code(), out.scale(), st);
      });
    }
  }
  return residual ? Coded::tuple(out.codes.object(), out.scales.object(), total.object(), 3) : out.pair();
}

at::ScalarType type_of(PyObject* o, at::ScalarType otherwise) {
  if (o == Py_None) return otherwise;
  if (!THPDtype_Check(o) || kind(reinterpret_cast<THPDtype*>(o)->scalar_type) < 0) bad("dtype must be fp32, bf16 or fp16");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// codes [n][k] with scales [n]
bool coded(const at::Tensor& c, const at::Tensor& s) {
  return c.dim() == 2 && c.scalar_type() == at::kChar && c.is_contiguous() && s.scalar_type() == at::kFloat && s.dim() == 1 &&
         s.size(0) == c.size(0) && s.is_contiguous();
}
at::Tensor on16(const at::Tensor& t) { return place(t) % 16 ? t.clone() : t; }

PyObject* dequantize(PyObject* const* a) {  // codes, scales, cols, dtype, out
  const at::Tensor &codes = tensor(a[0]), &scales = tensor(a[1]);
  const int dev = cuda_of(codes);
  if (dev < 0 || cuda_of(scales) != dev) bad(kDevice);
  if (!coded(codes, scales)) bad("dequantize_q8 takes contiguous int8 codes [rows][columns rounded up to 16] and fp32 scales [rows]");
  const int64_t n = codes.size(0), pitch = codes.size(1);
  long long cols = pitch;
  if (a[2] != Py_None) {
    cols = PyLong_AsLongLong(a[2]);
    if (cols == -1 && PyErr_Occurred()) throw python_error();
  }
  if (cols < 1 || cols > pitch || (cols + 15) / 16 * 16 != pitch) bad("codes must hold cols columns, rounded up to 16");
  const at::ScalarType type = type_of(a[3], at::kFloat);
  const Out out = output(a[4], {n, cols}, type, codes, "out must be contiguous [rows][cols] of dtype on the codes' device");
  if (n) {
    const at::Tensor c = on16(codes);
    launch("s2_dequantize_q8", dev, [&](CUstream_st* st) {
      return s2_dequantize_q8(static_cast<const int8_t*>(c.data_ptr()), static_cast<const float*>(scales.data_ptr()), n, whole(cols),
                              out.t.data_ptr(), kind(type), st);
    });
  }
  PyObject* o = out.object();
  if (!o) throw python_error();
  return o;
}

PyObject* matmul(PyObject* const* a) {  // x_codes, x_scales, codes, scales, dtype, out
  const at::Tensor &x = tensor(a[0]), &xs = tensor(a[1]), &w = tensor(a[2]), &ws = tensor(a[3]);
  const int dev = cuda_of(x);
  if (dev < 0 || cuda_of(xs) != dev || cuda_of(w) != dev || cuda_of(ws) != dev) bad(kDevice);
  if (x.dim() != 2 || w.dim() != 2 || x.scalar_type() != at::kChar || w.scalar_type() != at::kChar || !x.is_contiguous() ||
      !w.is_contiguous())
    bad("q8_matmul takes contiguous int8 codes [n][k] and [m][k]");
  const int64_t n = x.size(0), k = x.size(1), m = w.size(0);
  if (w.size(1) != k || !k || k % 16) bad("both operands' codes must have the same columns, a multiple of 16");
  if (!coded(x, xs) || !coded(w, ws)) bad("scales must be contiguous fp32 [n] and [m]");
  const at::ScalarType type = type_of(a[4], at::kBFloat16);
  const Out out = output(a[5], {n, m}, type, x, "out must be contiguous [n][m] of dtype, on the operands' device");
  if (n && m) {
    const at::Tensor c = on16(x), d = on16(w);
    launch("s2_q8_matmul", dev, [&](CUstream_st* st) {
      return s2_q8_matmul(whole(n), static_cast<const int8_t*>(c.data_ptr()), static_cast<const float*>(xs.data_ptr()),
                          static_cast<const int8_t*>(d.data_ptr()), static_cast<const float*>(ws.data_ptr()), whole(m), whole(k),
                          out.t.data_ptr(), kind(type), st);
    });
  }
  PyObject* o = out.object();
  if (!o) throw python_error();
  return o;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments were expected", kArgs);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const Bad& b) {
    PyErr_SetString(PyExc_ValueError, b.what);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(s2_error, type);
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<kCall, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<quantize, 3>("quantize_q8"),
                         method<dequantize, 5>("dequantize_q8"),
                         method<norm, 7>("rms_norm_q8"),
                         method<swiglu, 3>("swiglu_q8"),
                         method<matmul, 6>("q8_matmul"),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
