// Python entry to the MXFP4 calls: takes torch tensors apart, checks them,
// allocates what the caller did not give, and passes raw pointers and the
// current stream to the C ABI.  Nothing is computed here.
//
// Compiled because these layers are short: a layer with few rows takes 5 to 8
// us on the GPU, and marshalling it in Python with ctypes took 10 us for one
// launch and 14 for two, 5 to 7 of them outside the library (here 4.7 and 7.7).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>
#include <string>
#include <utility>

#include "svdq.h"

namespace {

PyObject* g_error = nullptr;                       // SvdqError(status, message)
PyObject *g_codes, *g_scales, *g_N, *g_K, *g_E;    // keys of a weight

// A refused call: TypeError, ValueError or SvdqError.
struct Refused {
  PyObject* type;
  std::string text;
  int status = 0;
};
struct PythonError {};   // already set

struct Held {            // a reference of our own
  PyObject* o;
  explicit Held(PyObject* reference) : o(reference) {}
  Held(Held&& h) noexcept : o(h.o) { h.o = nullptr; }
  Held& operator=(Held&& h) noexcept {
    std::swap(o, h.o);
    return *this;
  }
  ~Held() { Py_XDECREF(o); }
};

[[noreturn]] void type_error(std::string s) { throw Refused{PyExc_TypeError, std::move(s)}; }
[[noreturn]] void value_error(std::string s) { throw Refused{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void svdq_error(int status, std::string s) { throw Refused{g_error, std::move(s), status}; }

std::string num(long long v) { return std::to_string(v); }

// The library's sizes are ints; a larger one must not reach it cut off.
int size_of(long long v, const char* name) {
  if (v < 0 || v > INT_MAX)
    svdq_error(SVDQ_ERR_UNSUPPORTED_SHAPE, std::string(name) + ": a size of " + num(v) + " is out of range");
  return (int)v;
}

enum : unsigned { kBf16 = 1, kFp16 = 2, kFp32 = 4 };
unsigned dtype_bit(at::ScalarType t) {
  return t == at::kBFloat16 ? kBf16 : t == at::kHalf ? kFp16 : t == at::kFloat ? kFp32 : 0;
}
int mx_dtype(at::ScalarType t) { return t == at::kBFloat16 ? MXFP4_BF16 : t == at::kHalf ? MXFP4_FP16 : MXFP4_FP32; }

// `allowed` is a set of the bits above.
at::ScalarType dtype_arg(PyObject* o, unsigned allowed) {
  if (!THPDtype_Check(o) || !(dtype_bit(reinterpret_cast<THPDtype*>(o)->scalar_type) & allowed))
    type_error(allowed & kFp32 ? "dtype must be torch.bfloat16 or torch.float32"
                               : "dtype must be torch.bfloat16 or torch.float16");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// A CUDA matrix whose rows are contiguous.
struct Matrix {
  const at::Tensor* t;
  at::ScalarType type;
  int rows, cols;
  long long ld;
  void* ptr;
};
Matrix matrix(PyObject* o, const char* name, unsigned allowed) {
  const at::Tensor* t = THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || !(dtype_bit(t->scalar_type()) & allowed) || t->dim() != 2 || !t->is_cuda())
    type_error(std::string(name) + " must be a 2-D CUDA tensor of torch.bfloat16" +
               (allowed & kFp16 ? ", torch.float16" : "") + (allowed & kFp32 ? ", torch.float32" : ""));
  const long long rows = t->size(0), cols = t->size(1);
  size_of(rows, name);
  size_of(cols, name);
  if (t->stride(1) != 1 && cols > 1) value_error(std::string(name) + ": the elements of a row must be contiguous");
  return {t, t->scalar_type(), (int)rows, (int)cols, rows > 1 ? t->stride(0) : cols, t->data_ptr()};
}

// Quantized rows: uint8 [rows, K/2].
struct Codes {
  const at::Tensor* t;
  int rows, K;
};
Codes codes_arg(PyObject* o) {
  const at::Tensor* t = THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || t->scalar_type() != at::kByte || t->dim() != 2 || !t->is_cuda())
    type_error("codes must be a 2-D CUDA uint8 tensor");
  return {t, size_of(t->size(0), "codes"), size_of(2 * t->size(1), "codes")};
}

// A contiguous tensor of `count` elements, or (None) a null pointer.
template <class T = void>
T* flat(PyObject* o, const char* name, at::Device dev, at::ScalarType type, long long count) {
  if (o == Py_None) return nullptr;
  const at::Tensor* t = THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || t->scalar_type() != type || t->device() != dev)
    type_error(std::string(name) + " must be a tensor of " + c10::toString(type) + " on " + dev.str());
  if (t->numel() != count || !t->is_contiguous())
    value_error(std::string(name) + " must be contiguous and have " + num(count) + " elements (it has " +
                num(t->numel()) + ")");
  return static_cast<T*>(t->data_ptr());
}
template <class T = void>
T* flat_given(PyObject* o, const char* name, at::Device dev, at::ScalarType type, long long count) {
  if (o == Py_None) type_error(std::string(name) + " must be a tensor");
  return flat<T>(o, name, dev, type, count);
}
int* status_arg(PyObject* o, at::Device dev) { return flat<int>(o, "dev_status", dev, at::kInt, 1); }

long long entry(PyObject* w, PyObject* key) {
  Held v{PyObject_GetItem(w, key)};
  if (!v.o) throw PythonError{};
  const long long n = PyLong_AsLongLong(v.o);
  if (n == -1 && PyErr_Occurred()) throw PythonError{};
  return n;
}
int width_of(PyObject* w, const char* name) { return size_of(entry(w, g_N), name); }

// Codes and scales of `matrices` weights [N, K] one behind the other: a
// mapping with "codes", "scales", "N", "K" and, unless it is one, "E".
struct Weight {
  Held codes_tensor, scales_tensor;
  const void *codes, *scales;
};
Weight weight(PyObject* w, const char* name, at::Device dev, int N, int K, long long matrices) {
  long long E = 1;
  if (PyMapping_HasKey(w, g_E)) E = entry(w, g_E);
  const long long wn = entry(w, g_N), wk = entry(w, g_K);
  if (wn != N || wk != K || E != matrices)
    svdq_error(SVDQ_ERR_UNSUPPORTED_SHAPE, std::string(name) + " is " + num(E) + " x [" + num(wn) + ", " + num(wk) +
                                               "], not " + num(matrices) + " x [" + num(N) + ", " + num(K) + "]");
  Held c{PyObject_GetItem(w, g_codes)};
  if (!c.o) throw PythonError{};
  Held s{PyObject_GetItem(w, g_scales)};
  if (!s.o) throw PythonError{};
  const long long tiles = matrices * (((long long)N + 127) / 128) * (((long long)K + 127) / 128);
  const void* codes = flat_given(c.o, "a weight's codes", dev, at::kByte, matrices * N * (K / 2));
  const void* scales = flat_given(s.o, "a weight's scales", dev, at::kByte, 512 * tiles);
  return {std::move(c), std::move(s), codes, scales};
}

// Rows of the call and the row index: row i is row i of x without one.
struct Index {
  int rows;
  const int* ptr;
};
Index index_arg(PyObject* o, int x_rows, at::Device dev) {
  if (o == Py_None) return {x_rows, nullptr};
  if (!THPVariable_Check(o)) type_error("row_index must be an int32 tensor");
  const long long n = THPVariable_Unpack(o).numel();
  size_of(n, "row_index");
  return {(int)n, flat<int>(o, "row_index", dev, at::kInt, n)};
}

struct Groups {
  int count;   // 0: no offsets
  const int* offsets;
};
Groups groups_arg(PyObject* o, at::Device dev, bool optional) {
  if (optional && o == Py_None) return {0, nullptr};
  const at::Tensor* t = THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || t->dim() != 1 || t->numel() < 2) type_error("offsets must be an int32 tensor [groups + 1]");
  const int n = size_of(t->numel(), "offsets");
  return {n - 1, flat<int>(o, "offsets", dev, at::kInt, n)};
}

long long scale_bytes(int rows, int K, int groups) {
  const long long n = groups ? mxfp4_grouped_scale_bytes(groups, rows, K) : mxfp4_scale_bytes(rows, K);
  if (n < 0)
    svdq_error(SVDQ_ERR_UNSUPPORTED_SHAPE,
               "unsupported shape rows=" + num(rows) + " K=" + num(K) + " groups=" + num(groups));
  return n;
}

// An output matrix: the caller's, checked, or a new one.
struct Out {
  at::Tensor made;
  PyObject* given = nullptr;
  void* ptr;
  long long ld;
  PyObject* result() {
    if (!given) return THPVariable_Wrap(std::move(made));
    Py_INCREF(given);
    return given;
  }
};
Out output(PyObject* o, const char* name, int rows, int cols, at::ScalarType type, at::Device dev, bool zero = false) {
  Out out;
  if (o == Py_None) {
    const auto options = at::TensorOptions().dtype(type).device(dev);
    out.made = zero ? at::zeros({rows, cols}, options) : at::empty({rows, cols}, options);
    out.ptr = out.made.data_ptr();
    out.ld = cols;
    return out;
  }
  const Matrix m = matrix(o, name, dtype_bit(type));
  if (m.rows != rows || m.cols != cols || m.t->device() != dev)
    value_error(std::string(name) + " must be [" + num(rows) + ", " + num(cols) + "] on " + dev.str());
  out.given = o;
  out.ptr = m.ptr;
  out.ld = m.ld;
  return out;
}

// Codes [rows, K/2] and their scales: the caller's pair, checked, or new.
struct Quantized {
  at::Tensor made_codes, made_scales;
  Held given_codes{nullptr}, given_scales{nullptr};
  void *codes, *scales;
  PyObject* result() {
    if (given_codes.o) return PyTuple_Pack(2, given_codes.o, given_scales.o);
    Held c{THPVariable_Wrap(std::move(made_codes))}, s{THPVariable_Wrap(std::move(made_scales))};
    return c.o && s.o ? PyTuple_Pack(2, c.o, s.o) : nullptr;
  }
};
Quantized quantized(PyObject* o, int rows, int K, int groups, at::Device dev) {
  const long long size = scale_bytes(rows, K, groups);
  Quantized q;
  if (o == Py_None) {
    const auto options = at::TensorOptions().dtype(at::kByte).device(dev);
    q.made_codes = at::empty({rows, K / 2}, options);
    q.made_scales = at::empty({size}, options);
    q.codes = q.made_codes.data_ptr();
    q.scales = q.made_scales.data_ptr();
    return q;
  }
  if (!PyTuple_Check(o) && !PyList_Check(o)) type_error("out must be a pair (codes, scales)");
  if (PySequence_Size(o) != 2) value_error("out must be a pair (codes, scales)");
  Held c{PySequence_GetItem(o, 0)}, s{PySequence_GetItem(o, 1)};
  if (!c.o || !s.o) throw PythonError{};
  q.codes = flat_given(c.o, "codes", dev, at::kByte, (long long)rows * (K / 2));
  q.scales = flat_given(s.o, "scales", dev, at::kByte, size);
  q.given_codes = std::move(c);
  q.given_scales = std::move(s);
  return q;
}

struct Workspace {
  at::Tensor made;   // until the launch; its memory belongs to the stream
  void* ptr = nullptr;
  long long bytes = 0;
};
Workspace workspace_arg(PyObject* o, long long need, at::Device dev) {
  if (need < 0) svdq_error(SVDQ_ERR_UNSUPPORTED_SHAPE, "unsupported shape");
  Workspace w;
  if (o == Py_None) {
    if (need > 0) {
      w.made = at::empty({need}, at::TensorOptions().dtype(at::kByte).device(dev));
      w.ptr = w.made.data_ptr();
      w.bytes = need;
    }
    return w;
  }
  const at::Tensor* t = THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
  if (!t || t->scalar_type() != at::kByte || t->device() != dev || !t->is_contiguous())
    type_error("workspace must be a contiguous uint8 tensor on " + dev.str());
  w.ptr = t->data_ptr();
  w.bytes = t->numel();
  return w;
}

// The library's call, without the interpreter's lock, on the current stream of
// the tensors' device.
template <class F>
void launch(at::Device dev, F&& call) {
  void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = call(stream);
  Py_END_ALLOW_THREADS;
  if (status == SVDQ_OK) return;
  const char* text = svdq_last_error();
  svdq_error(status, text && *text ? text : svdq_status_string(status));
}

// Runs a binding and turns what it throws into Python's exceptions.
template <int kArgs, PyObject* (*kFn)(PyObject* const*)>
PyObject* entry_point(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return kFn(args);
  } catch (const PythonError&) {
  } catch (const Refused& r) {
    if (r.status == 0) {
      PyErr_SetString(r.type, r.text.c_str());
    } else {
      Held e{PyObject_CallFunction(r.type, "is", r.status, r.text.c_str())};
      if (e.o) PyErr_SetObject(r.type, e.o);
    }
  } catch (...) {   // torch's own, out of memory among them
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// ------------------------------------------------------------------ bindings
// (x, offsets, row_index, out, dev_status)
PyObject* quantize(PyObject* const* a) {
  const Matrix x = matrix(a[0], "x", kBf16 | kFp16 | kFp32);
  const at::Device dev = x.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const Index i = index_arg(a[2], x.rows, dev);
  const Groups g = groups_arg(a[1], dev, true);
  Quantized q = quantized(a[3], i.rows, x.cols, g.count, dev);
  int* status = status_arg(a[4], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_quantize(mx_dtype(x.type), i.rows, x.cols, x.ptr, x.ld, i.ptr, x.rows, g.count, g.offsets, q.codes,
                          q.scales, status, stream);
  });
  return q.result();
}

// (codes, scales, offsets, dtype, out, dev_status)
PyObject* dequantize(PyObject* const* a) {
  const Codes c = codes_arg(a[0]);
  const at::Device dev = c.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const at::ScalarType type = dtype_arg(a[3], kBf16 | kFp32);
  const Groups g = groups_arg(a[2], dev, true);
  const void* codes = flat_given(a[0], "codes", dev, at::kByte, (long long)c.rows * (c.K / 2));
  const void* scales = flat_given(a[1], "scales", dev, at::kByte, scale_bytes(c.rows, c.K, g.count));
  Out out = output(a[4], "out", c.rows, c.K, type, dev, g.count > 0);
  int* status = status_arg(a[5], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_dequantize(mx_dtype(type), c.rows, c.K, codes, scales, g.count, g.offsets, out.ptr, out.ld, status,
                            stream);
  });
  return out.result();
}

// (codes, scales, offsets, w, bias, dtype, y, dev_status)
PyObject* grouped_gemm(PyObject* const* a) {
  const Codes c = codes_arg(a[0]);
  const at::Device dev = c.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const at::ScalarType type = dtype_arg(a[5], kBf16 | kFp16);
  const int N = width_of(a[3], "w");
  const Groups g = groups_arg(a[2], dev, true);
  const long long matrices = g.count ? g.count : 1;
  const Weight w = weight(a[3], "w", dev, N, c.K, matrices);
  const void* codes = flat_given(a[0], "codes", dev, at::kByte, (long long)c.rows * (c.K / 2));
  const void* scales = flat_given(a[1], "scales", dev, at::kByte, scale_bytes(c.rows, c.K, g.count));
  const void* bias = flat(a[4], "bias", dev, type, matrices * N);
  Out y = output(a[6], "y", c.rows, N, type, dev);
  int* status = status_arg(a[7], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_grouped_gemm(mx_dtype(type), g.count, c.rows, N, c.K, g.offsets, codes, scales, w.codes, w.scales,
                              bias, y.ptr, y.ld, status, stream);
  });
  return y.result();
}

// (x, w, bias, y, workspace, dev_status)
PyObject* linear(PyObject* const* a) {
  const Matrix x = matrix(a[0], "x", kBf16 | kFp16);
  const at::Device dev = x.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const int N = width_of(a[1], "w");
  const Weight w = weight(a[1], "w", dev, N, x.cols, 1);
  const void* bias = flat(a[2], "bias", dev, x.type, N);
  Out y = output(a[3], "y", x.rows, N, x.type, dev);
  const Workspace ws = workspace_arg(a[4], mxfp4_workspace_bytes(0, x.rows, x.cols), dev);
  int* status = status_arg(a[5], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_linear(mx_dtype(x.type), x.rows, N, x.cols, x.ptr, x.ld, w.codes, w.scales, bias, y.ptr, y.ld, ws.ptr,
                        ws.bytes, status, stream);
  });
  return y.result();
}

// (x, offsets, w, row_index, bias, y, workspace, dev_status)
PyObject* grouped_linear(PyObject* const* a) {
  const Matrix x = matrix(a[0], "x", kBf16 | kFp16);
  const at::Device dev = x.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const Index i = index_arg(a[3], x.rows, dev);
  const int N = width_of(a[2], "w");
  const Groups g = groups_arg(a[1], dev, false);
  const Weight w = weight(a[2], "w", dev, N, x.cols, g.count);
  const void* bias = flat(a[4], "bias", dev, x.type, (long long)g.count * N);
  Out y = output(a[5], "y", i.rows, N, x.type, dev);
  const Workspace ws = workspace_arg(a[6], mxfp4_workspace_bytes(g.count, i.rows, x.cols), dev);
  int* status = status_arg(a[7], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_grouped_linear(mx_dtype(x.type), g.count, i.rows, N, x.cols, x.ptr, x.ld, i.ptr, x.rows, g.offsets,
                                w.codes, w.scales, bias, y.ptr, y.ld, ws.ptr, ws.bytes, status, stream);
  });
  return y.result();
}

// (codes, scales, offsets, w, bias, dtype, out, dev_status)
PyObject* grouped_gemm_swiglu_quant(PyObject* const* a) {
  const Codes c = codes_arg(a[0]);
  const at::Device dev = c.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const at::ScalarType type = dtype_arg(a[5], kBf16 | kFp16);
  const int width = width_of(a[3], "w");
  const Groups g = groups_arg(a[2], dev, false);
  const Weight w = weight(a[3], "w", dev, width, c.K, 2ll * g.count);
  const void* codes = flat_given(a[0], "codes", dev, at::kByte, (long long)c.rows * (c.K / 2));
  const void* scales = flat_given(a[1], "scales", dev, at::kByte, scale_bytes(c.rows, c.K, g.count));
  const void* bias = flat(a[4], "bias", dev, type, 2ll * g.count * width);
  Quantized h = quantized(a[6], c.rows, width, g.count, dev);
  int* status = status_arg(a[7], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_grouped_gemm_swiglu_quant(mx_dtype(type), g.count, c.rows, width, c.K, g.offsets, codes, scales,
                                           w.codes, w.scales, bias, h.codes, h.scales, status, stream);
  });
  return h.result();
}

// (x, offsets, w_up, w_down, row_index, up_bias, down_bias, y, workspace, dev_status)
PyObject* grouped_mlp_swiglu(PyObject* const* a) {
  const Matrix x = matrix(a[0], "x", kBf16 | kFp16);
  const at::Device dev = x.t->device();
  const c10::cuda::CUDAGuard guard(dev);
  const Index i = index_arg(a[4], x.rows, dev);
  const int width = width_of(a[2], "w_up");
  const Groups g = groups_arg(a[1], dev, false);
  const Weight up = weight(a[2], "w_up", dev, width, x.cols, 2ll * g.count);
  const Weight down = weight(a[3], "w_down", dev, x.cols, width, g.count);
  const void* up_bias = flat(a[5], "up_bias", dev, x.type, 2ll * g.count * width);
  const void* down_bias = flat(a[6], "down_bias", dev, x.type, (long long)g.count * x.cols);
  Out y = output(a[7], "y", i.rows, x.cols, x.type, dev);
  const Workspace ws = workspace_arg(a[8], mxfp4_mlp_workspace_bytes(g.count, i.rows, x.cols, width), dev);
  int* status = status_arg(a[9], dev);
  launch(dev, [&](void* stream) {
    return mxfp4_grouped_mlp_swiglu(mx_dtype(x.type), g.count, i.rows, x.cols, width, x.ptr, x.ld, i.ptr, x.rows,
                                    g.offsets, up.codes, up.scales, up_bias, down.codes, down.scales, down_bias, y.ptr,
                                    y.ld, ws.ptr, ws.bytes, status, stream);
  });
  return y.result();
}

// The class of the library's errors.
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

#define MX_ENTRY(name, args) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry_point<args, name>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {
    MX_ENTRY(quantize, 5),
    MX_ENTRY(dequantize, 6),
    MX_ENTRY(grouped_gemm, 8),
    MX_ENTRY(linear, 6),
    MX_ENTRY(grouped_linear, 8),
    MX_ENTRY(grouped_gemm_swiglu_quant, 8),
    MX_ENTRY(grouped_mlp_swiglu, 10),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_mxfp4", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mxfp4() {
  struct {
    PyObject** key;
    const char* name;
  } keys[] = {{&g_codes, "codes"}, {&g_scales, "scales"}, {&g_N, "N"}, {&g_K, "K"}, {&g_E, "E"}};
  for (auto& k : keys)
    if (!(*k.key = PyUnicode_InternFromString(k.name))) return nullptr;
  PyObject* const module = PyModule_Create(&g_module);
  if (module && PyModule_AddStringConstant(module, "built_for_torch", BUILT_FOR_TORCH) != 0) {
    Py_DECREF(module);
    return nullptr;
  }
  return module;
}
