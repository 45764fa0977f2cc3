// Python binding of the 8-bit activation calls (module _act8): argument
// checks, allocation of results and scratch, and the call of the C entry
// point, nothing computed.  The smallest of these calls take 2 to 7 us on the
// device; through ctypes and Python-level checks the host needed 10 to 16 us
// for each, here 4 to 8.
//
// Every function takes positional arguments only (api.py gives them names and
// defaults) and follows the same order: check, allocate (results on the
// current stream, and kept for the call's stream; scratch on the call's
// stream), call on the tensors' device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <algorithm>
#include <memory>
#include <string>
#include <vector>
#include "shampoo4.h"

namespace {

PyObject* g_check = nullptr;       // _lib.check(name, status): raises Shampoo4Error

struct Refused {                   // a Python exception is set
  Refused(PyObject* type, const std::string& text) { PyErr_SetString(type, text.c_str()); }
  Refused() {}
};

[[noreturn]] void type_error(const std::string& s) { throw Refused(PyExc_TypeError, s); }
[[noreturn]] void value_error(const std::string& s) { throw Refused(PyExc_ValueError, s); }

std::string shape_text(int64_t r, int64_t c) { return "(" + std::to_string(r) + ", " + std::to_string(c) + ")"; }

int32_t dtype_code(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kFloat: return ACT8_FP32;
    case at::kBFloat16: return ACT8_BF16;
    case at::kHalf: return ACT8_FP16;
    default: type_error(std::string(name) + " must be float32, bfloat16 or float16, not " + c10::toString(t));
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) type_error(std::string(name) + " must be a CUDA tensor");
  return t;
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

int64_t padded(int64_t cols) { return (cols + 15) / 16 * 16; }

int64_t groups_of(int64_t cols, int64_t group) {
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
    value_error("group must be 0, 32, 64, 128 or 256");
  if (cols == 0) return 0;
  return group == 0 ? 1 : (cols + group - 1) / group;
}

// A float matrix: 2-D, unit column stride.
struct Mat {
  void* p;
  int32_t dtype;
  int64_t rows, cols, ld;
  c10::Device device{c10::kCUDA};
};
Mat mat(const at::Tensor& t, const char* name) {
  Mat m;
  m.dtype = dtype_code(t.scalar_type(), name);
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    value_error(std::string(name) + " must be 2-D with unit column stride");
  m.rows = t.size(0);
  m.cols = t.size(1);
  // a single row has no stride of its own: any that keeps its alignment
  m.ld = m.rows > 1 ? t.stride(0) : padded(m.cols);
  m.p = t.data_ptr();
  m.device = t.device();
  return m;
}
Mat mat(PyObject* o, const char* name) { return mat(tensor(o, name), name); }
void same_device(c10::Device a, c10::Device b, const char* name) {
  if (a != b) value_error(std::string(name) + " is on " + a.str() + ", not on " + b.str());
}
void want_shape(const Mat& m, int64_t rows, int64_t cols, const char* name) {
  if (m.rows != rows || m.cols != cols)
    value_error(std::string(name) + ": shape " + shape_text(m.rows, m.cols) + " != " + shape_text(rows, cols));
}

at::Tensor empty(int64_t rows, int64_t cols, int64_t ld, at::ScalarType t, c10::Device d) {
  return at::empty_strided({rows, cols}, {ld, 1}, at::TensorOptions().dtype(t).device(d));
}

// Stored codes and their scales.
struct Codes {
  int8_t* p;
  int64_t rows, cols, ld;
  float* scales;
  c10::Device device{c10::kCUDA};
};
Codes codes(PyObject* oc, PyObject* os, int64_t group, const char* name) {
  const std::string n(name);
  if (!THPVariable_Check(oc)) type_error(n + " codes must be a 2-D CUDA int8 tensor");
  const at::Tensor& c = THPVariable_Unpack(oc);
  if (!c.is_cuda() || c.scalar_type() != at::kChar || c.dim() != 2)
    type_error(n + " codes must be a 2-D CUDA int8 tensor");
  if (!THPVariable_Check(os)) type_error(n + " scales must be a CUDA float32 tensor");
  const at::Tensor& s = THPVariable_Unpack(os);
  if (!s.is_cuda() || s.scalar_type() != at::kFloat) type_error(n + " scales must be a CUDA float32 tensor");
  Codes k;
  k.rows = c.size(0);
  k.cols = c.size(1);
  if (k.cols > 1 && c.stride(1) != 1) value_error(n + " codes must have unit column stride");
  const int64_t groups = groups_of(k.cols, group);
  if (s.dim() != 2 || s.size(0) != k.rows || s.size(1) != groups || !s.is_contiguous())
    value_error(n + " scales must be a contiguous " + std::to_string(k.rows) + " x " + std::to_string(groups) +
                " tensor");
  k.device = c.device();
  if (s.device() != k.device) value_error(n + " codes and scales must be on one device");
  k.ld = k.rows > 1 ? c.stride(0) : padded(k.cols);
  k.p = static_cast<int8_t*>(c.data_ptr());
  k.scales = static_cast<float*>(s.data_ptr());
  if (k.rows && k.cols && ((k.ld | int64_t(reinterpret_cast<uintptr_t>(k.p))) & 15))
    value_error(n + " codes must be 16-byte aligned with rows a multiple of 16 bytes apart");
  return k;
}
Codes codes_on(PyObject* oc, PyObject* os, int64_t group, const char* name, c10::Device d) {
  const Codes k = codes(oc, os, group, name);
  same_device(k.device, d, name);
  return k;
}

// Fresh codes (rows padded to 16 bytes) and scales.
struct Store {
  at::Tensor codes, scales;
  Codes k;
};
Store store(int64_t rows, int64_t cols, int64_t group, c10::Device d) {
  Store s;
  const int64_t groups = groups_of(cols, group), ld = padded(cols);
  s.codes = empty(rows, cols, ld, at::kChar, d);
  s.scales = empty(rows, groups, groups, at::kFloat, d);
  s.k.p = static_cast<int8_t*>(s.codes.data_ptr());
  s.k.rows = rows;
  s.k.cols = cols;
  s.k.ld = ld;
  s.k.scales = static_cast<float*>(s.scales.data_ptr());
  s.k.device = d;
  return s;
}

// The result: the caller's tensor, or a fresh one of `t`.
struct Out {
  at::Tensor made;
  PyObject* given = nullptr;
  Mat m;
  PyObject* object() const {           // a new reference
    if (!given) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};
Out result(PyObject* o, int64_t rows, int64_t cols, at::ScalarType t, c10::Device d, const char* name) {
  Out r;
  if (o == Py_None) {
    r.m.dtype = dtype_code(t, "dtype");
    r.made = empty(rows, cols, cols, t, d);
    r.m.p = r.made.data_ptr();
    r.m.rows = rows;
    r.m.cols = cols;
    r.m.ld = rows > 1 ? cols : padded(cols);
    r.m.device = d;
    return r;
  }
  r.given = o;
  r.m = mat(o, name);
  want_shape(r.m, rows, cols, name);
  same_device(r.m.device, d, name);
  return r;
}

at::ScalarType scalar_type(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) type_error(std::string(name) + " must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  dtype_code(t, name);
  return t;
}

// Pointer of an optional contiguous vector of n elements.
void* vec(PyObject* o, int64_t n, std::initializer_list<at::ScalarType> types, const char* what, const char* name,
          c10::Device d) {
  if (o == Py_None) return nullptr;
  bool ok = THPVariable_Check(o);
  if (ok) {
    const at::Tensor& t = THPVariable_Unpack(o);
    ok = t.is_cuda() && t.is_contiguous() && t.numel() == n && t.device() == d &&
         std::find(types.begin(), types.end(), t.scalar_type()) != types.end();
    if (ok) return t.data_ptr();
  }
  type_error(std::string(name) + " must be a contiguous " + what + " tensor of " + std::to_string(n) + " on " +
             d.str());
}
float* bias_of(PyObject* o, int64_t n, c10::Device d) {
  return static_cast<float*>(vec(o, n, {at::kFloat}, "float32", "bias", d));
}
uint32_t* flags_of(PyObject* o, c10::Device d) {
  return static_cast<uint32_t*>(vec(o, 1, {at::kInt, at::kUInt32}, "int32", "flags", d));
}

// The tensors' device, current for the call, and the stream: the given one,
// or the device's current one.
struct Where {
  c10::cuda::OptionalCUDAGuard guard;
  c10::Device device;
  cudaStream_t st;
  bool given;
  Where(c10::Device d, PyObject* stream) : device(d), given(stream != Py_None) {
    if (c10::cuda::current_device() != d.index()) guard.set_device(d);
    if (!given) {
      st = c10::cuda::getCurrentCUDAStream(d.index()).stream();
      return;
    }
    PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
    if (!raw) throw Refused();
    st = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
    Py_DECREF(raw);
    if (!st && PyErr_Occurred()) throw Refused();
  }
  // A fresh result dropped while this stream still writes it stays allocated.
  void keep(const at::Tensor& t) const {
    if (given && t.defined()) t.record_stream(c10::cuda::getStreamFromExternal(st, device.index()).unwrap());
  }
  shampoo4_stream_t stream() const { return reinterpret_cast<shampoo4_stream_t>(st); }
  // Scratch that the caching allocator keeps for the work on this stream.
  at::Tensor scratch(int64_t bytes) const {
    const auto make = [&] { return at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(device)); };
    if (!given) return make();
    const c10::cuda::CUDAStreamGuard on(c10::cuda::getStreamFromExternal(st, device.index()));
    return make();
  }
};

void check(const char* fn, shampoo4_status st) {
  if (st == SHAMPOO4_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "si", fn, int(st));
  Py_XDECREF(r);
  throw Refused();
}

void want_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("expected " + std::to_string(want) + " arguments");
}

int64_t inner_of(int64_t inner, const Codes& w, const char* what) {
  if (inner != w.cols)
    value_error(std::string(what) + ": inner sizes " + std::to_string(inner) + " and " + std::to_string(w.cols) +
                " differ");
  if (inner > (int64_t(1) << 17)) value_error(std::string(what) + ": inner size " + std::to_string(inner) + " > 2^17");
  return w.rows;
}

// A call that turns what the checks threw, and any C++ exception, into a
// Python exception.
template <class F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}

// pack(x, group, codes, scales, stream) -> (codes, scales)
PyObject* pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 5);
    const Mat x = mat(a[0], "x");
    const int64_t group = integer(a[1], "group");
    if ((a[2] == Py_None) != (a[3] == Py_None)) value_error("give both codes and scales, or neither");
    Store s;
    Codes k;
    if (a[2] == Py_None) {
      s = store(x.rows, x.cols, group, x.device);
      k = s.k;
    } else {
      k = codes_on(a[2], a[3], group, "x", x.device);
      if (k.rows != x.rows || k.cols != x.cols)
        value_error("codes: shape " + shape_text(k.rows, k.cols) + " != " + shape_text(x.rows, x.cols));
    }
    const Where w(x.device, a[4]);
    check("act8_pack", act8_pack(x.p, x.dtype, x.rows, x.cols, x.ld, int32_t(group), k.p, k.ld, k.scales, w.stream()));
    w.keep(s.codes);
    w.keep(s.scales);
    if (a[2] != Py_None) return PyTuple_Pack(2, a[2], a[3]);
    return pair(THPVariable_Wrap(s.codes), THPVariable_Wrap(s.scales));
  });
}

// unpack(codes, scales, group, dtype, out, stream) -> out
PyObject* unpack(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 6);
    const int64_t group = integer(a[2], "group");
    const Codes k = codes(a[0], a[1], group, "x");
    const Out o = result(a[4], k.rows, k.cols, scalar_type(a[3], "dtype"), k.device, "out");
    const Where w(k.device, a[5]);
    check("act8_unpack", act8_unpack(k.p, k.ld, k.scales, k.rows, k.cols, int32_t(group), o.m.p, o.m.dtype, o.m.ld,
                                     w.stream()));
    w.keep(o.made);
    return o.object();
  });
}

// matmul(x_codes, x_scales, w_codes, w_scales, bias, dtype, out, flags, stream) -> out
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 9);
    const Codes x = codes(a[0], a[1], 0, "x"), k = codes_on(a[2], a[3], 0, "w", x.device);
    const int64_t outs = inner_of(x.cols, k, "act8_matmul");
    const Out o = result(a[6], x.rows, outs, scalar_type(a[5], "dtype"), x.device, "out");
    const float* bias = bias_of(a[4], outs, x.device);
    uint32_t* flags = flags_of(a[7], x.device);
    const Where w(x.device, a[8]);
    check("act8_matmul", act8_matmul(x.p, x.ld, x.scales, k.p, k.ld, k.scales, bias, x.rows, outs, x.cols, o.m.p,
                                     o.m.dtype, o.m.ld, flags, w.stream()));
    w.keep(o.made);
    return o.object();
  });
}

// linear(x, w_codes, w_scales, bias, out, checkpoint, flags, stream) -> out, or (out, codes, scales)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 8);
    const at::Tensor& tx = tensor(a[0], "x");
    const Mat x = mat(tx, "x");
    const Codes k = codes_on(a[1], a[2], 0, "w", x.device);
    const int64_t outs = inner_of(x.cols, k, "act8_linear");
    const Out o = result(a[4], x.rows, outs, tx.scalar_type(), x.device, "out");
    const float* bias = bias_of(a[3], outs, x.device);
    uint32_t* flags = flags_of(a[6], x.device);
    const int keep = PyObject_IsTrue(a[5]);
    if (keep < 0) throw Refused();
    const Where w(x.device, a[7]);
    Store s;
    at::Tensor work;
    Codes c;
    if (keep) {
      s = store(x.rows, x.cols, 0, x.device);
      c = s.k;
    } else {                             // scratch of this call: codes, then scales
      c.ld = padded(x.cols);
      work = w.scratch(x.rows * c.ld + 4 * x.rows);
      c.p = static_cast<int8_t*>(work.data_ptr());
      c.scales = reinterpret_cast<float*>(c.p + x.rows * c.ld);
    }
    check("act8_linear", act8_linear(x.p, x.dtype, x.ld, k.p, k.ld, k.scales, bias, x.rows, outs, x.cols, c.p, c.ld,
                                     c.scales, o.m.p, o.m.dtype, o.m.ld, flags, w.stream()));
    w.keep(o.made);
    w.keep(s.codes);
    w.keep(s.scales);
    if (!keep) return o.object();
    PyObject* r = PyTuple_New(3);
    if (!r) throw Refused();
    PyTuple_SET_ITEM(r, 0, o.object());
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(s.codes));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(s.scales));
    return r;
  });
}

// grad(weight, dy, codes, scales, group, dtype, out, accumulate, flags, stream) -> out
PyObject* grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 10);
    const bool weight = a[0] == Py_True;
    const int64_t group = integer(a[4], "group");
    const at::Tensor& tdy = tensor(a[1], "dy");
    const Mat dy = mat(tdy, "dy");
    const Codes k = codes_on(a[2], a[3], group, weight ? "x" : "w", dy.device);
    if (weight && dy.rows != k.rows) value_error("dy and x must have the same number of rows");
    if (!weight && dy.cols != k.rows) value_error("dy's columns must match w's rows");
    const int add = PyObject_IsTrue(a[7]);
    if (add < 0) throw Refused();
    if (add && a[6] == Py_None) value_error("accumulate needs out");
    const at::ScalarType t = a[5] == Py_None ? tdy.scalar_type() : scalar_type(a[5], "dtype");
    const Out o = result(a[6], weight ? dy.cols : dy.rows, k.cols, t, dy.device, "out");
    uint32_t* flags = flags_of(a[8], dy.device);
    const Where w(dy.device, a[9]);
    size_t bytes = 0;
    check("act8_grad_workspace", act8_grad_workspace(weight, dy.dtype, o.m.dtype, dy.rows, dy.cols, k.cols,
                                                     int32_t(group), &bytes));
    const at::Tensor work = w.scratch(int64_t(bytes));
    if (weight)
      check("act8_weight_grad", act8_weight_grad(dy.p, dy.dtype, dy.ld, k.p, k.ld, k.scales, int32_t(group), dy.rows,
                                                 dy.cols, k.cols, o.m.p, o.m.dtype, o.m.ld, add, work.data_ptr(),
                                                 bytes, flags, w.stream()));
    else
      check("act8_input_grad", act8_input_grad(dy.p, dy.dtype, dy.ld, k.p, k.ld, k.scales, dy.rows, dy.cols, k.cols,
                                               o.m.p, o.m.dtype, o.m.ld, add, work.data_ptr(), bytes, flags,
                                               w.stream()));
    w.keep(o.made);
    return o.object();
  });
}

// The items of a list or tuple of n.
struct Items {
  PyObject* fast;
  Items(PyObject* o, Py_ssize_t n, const char* name) : fast(PySequence_Fast(o, name)) {
    if (!fast) throw Refused();
    if (PySequence_Fast_GET_SIZE(fast) != n) {
      Py_DECREF(fast);
      value_error("expected " + std::to_string(n) + " " + name);
    }
  }
  Items(const Items&) = delete;
  ~Items() { Py_DECREF(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// weight_grads(handle, state, shapes, dys, inputs, group, grads, accumulate, stream) -> grads (a new list, or the given one)
PyObject* weight_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 9);
    const auto h = static_cast<shampoo4_handle>(PyLong_AsVoidPtr(a[0]));
    if (!h) throw Refused();
    const c10::Device device = tensor(a[1], "state").device();
    const Py_ssize_t count = PyObject_Length(a[2]);
    if (count < 0) throw Refused();
    const Items shapes(a[2], count, "shapes"), dys(a[3], count, "dys"), inputs(a[4], count, "inputs");
    const int64_t group = integer(a[5], "group");
    const int add = PyObject_IsTrue(a[7]);
    if (add < 0) throw Refused();
    const bool given = a[6] != Py_None;
    if (add && !given) value_error("accumulate needs grads");
    std::vector<shampoo4_layer> layers;
    std::vector<at::Tensor> made;
    std::vector<float*> grads;
    std::vector<int64_t> ld;
    const std::unique_ptr<Items> old(given ? new Items(a[6], count, "grads") : nullptr);
    for (Py_ssize_t i = 0; i < count; ++i) {
      const Items shape(shapes[i], 2, "sizes of a shape"), input(inputs[i], 2, "tensors (codes, scales) of an input");
      const int64_t out = integer(shape[0], "shape"), inner = integer(shape[1], "shape");
      const Mat dy = mat(dys[i], "dys");
      same_device(dy.device, device, "dys");
      const Codes k = codes_on(input[0], input[1], group, "inputs", device);
      want_shape(dy, k.rows, out, "dys");
      if (k.cols != inner) value_error("inputs: " + std::to_string(k.cols) + " columns, not " + std::to_string(inner));
      layers.push_back({dy.p, dy.dtype, dy.ld, k.p, k.ld, k.scales, k.rows});
      if (!given) continue;
      const at::Tensor& t = tensor((*old)[i], "grads");
      if (t.scalar_type() != at::kFloat) type_error("grads must be float32");
      const Mat g = mat(t, "grads");
      want_shape(g, out, inner, "grads");
      same_device(g.device, device, "grads");
      grads.push_back(static_cast<float*>(g.p));
      ld.push_back(g.rows > 1 ? g.ld : std::max(g.ld, g.cols));
    }
    const Where w(device, a[8]);
    for (Py_ssize_t i = 0; i < count && !given; ++i) {
      const Items shape(shapes[i], 2, "sizes of a shape");
      const int64_t out = integer(shape[0], "shape"), inner = integer(shape[1], "shape");
      made.push_back(empty(out, inner, inner, at::kFloat, device));
      grads.push_back(static_cast<float*>(made.back().data_ptr()));
      ld.push_back(inner);
    }
    size_t bytes = 0;
    check("shampoo4_weight_grads_workspace", shampoo4_weight_grads_workspace(h, layers.data(), int32_t(group), &bytes));
    const at::Tensor work = w.scratch(int64_t(bytes));
    check("shampoo4_weight_grads", shampoo4_weight_grads(h, layers.data(), int32_t(group), grads.data(), ld.data(), add,
                                                         work.data_ptr(), bytes, w.stream()));
    for (const at::Tensor& t : made) w.keep(t);
    if (given) {
      Py_INCREF(a[6]);
      return a[6];
    }
    PyObject* r = PyList_New(count);
    if (!r) throw Refused();
    for (Py_ssize_t i = 0; i < count; ++i) PyList_SET_ITEM(r, i, THPVariable_Wrap(made[size_t(i)]));
    return r;
  });
}

// swiglu(gate, up, group, out, stream) -> (h, (gate codes, gate scales, up codes, up scales))
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 5);
    const at::Tensor& tg = tensor(a[0], "gate");
    const Mat g = mat(tg, "gate"), u = mat(a[1], "up");
    want_shape(u, g.rows, g.cols, "up");
    same_device(u.device, g.device, "up");
    const int64_t group = integer(a[2], "group");
    const Out o = result(a[3], g.rows, g.cols, tg.scalar_type(), g.device, "out");
    if (u.dtype != g.dtype || o.m.dtype != g.dtype) type_error("gate, up and out must have one type");
    const Store sg = store(g.rows, g.cols, group, g.device), su = store(g.rows, g.cols, group, g.device);
    const Where w(g.device, a[4]);
    check("act8_swiglu", act8_swiglu(g.p, g.ld, u.p, u.ld, g.dtype, g.rows, g.cols, int32_t(group), o.m.p, o.m.ld,
                                     sg.k.p, sg.k.ld, sg.k.scales, su.k.p, su.k.ld, su.k.scales, w.stream()));
    w.keep(o.made);
    for (const Store* s : {&sg, &su}) {
      w.keep(s->codes);
      w.keep(s->scales);
    }
    PyObject* kept = PyTuple_New(4);
    if (!kept) throw Refused();
    PyTuple_SET_ITEM(kept, 0, THPVariable_Wrap(sg.codes));
    PyTuple_SET_ITEM(kept, 1, THPVariable_Wrap(sg.scales));
    PyTuple_SET_ITEM(kept, 2, THPVariable_Wrap(su.codes));
    PyTuple_SET_ITEM(kept, 3, THPVariable_Wrap(su.scales));
    return pair(o.object(), kept);
  });
}

// swiglu_backward(dh, kept, group, dgate, dup, stream) -> (dgate, dup)
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 6);
    const at::Tensor& td = tensor(a[0], "dh");
    const Mat d = mat(td, "dh");
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 4)
      type_error("kept must be the four tensors of act8_swiglu");
    const int64_t group = integer(a[2], "group");
    const Codes g = codes_on(PyTuple_GET_ITEM(a[1], 0), PyTuple_GET_ITEM(a[1], 1), group, "gate", d.device);
    const Codes u = codes_on(PyTuple_GET_ITEM(a[1], 2), PyTuple_GET_ITEM(a[1], 3), group, "up", d.device);
    want_shape(d, g.rows, g.cols, "dh");
    if (u.rows != g.rows || u.cols != g.cols) value_error("gate and up codes differ in shape");
    const Out og = result(a[3], d.rows, d.cols, td.scalar_type(), d.device, "dgate");
    const Out ou = result(a[4], d.rows, d.cols, td.scalar_type(), d.device, "dup");
    if (og.m.dtype != d.dtype || ou.m.dtype != d.dtype) type_error("dh, dgate and dup must have one type");
    const Where w(d.device, a[5]);
    check("act8_swiglu_backward",
          act8_swiglu_backward(d.p, d.ld, d.dtype, g.p, g.ld, g.scales, u.p, u.ld, u.scales, d.rows, d.cols,
                               int32_t(group), og.m.p, og.m.ld, ou.m.p, ou.m.ld, w.stream()));
    w.keep(og.made);
    w.keep(ou.made);
    return pair(og.object(), ou.object());
  });
}

// set_check(function): what turns a status into an exception
PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XDECREF(g_check);
  g_check = f;
  Py_RETURN_NONE;
}

#define S4_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {S4_FAST(pack), S4_FAST(unpack), S4_FAST(matmul), S4_FAST(linear), S4_FAST(grad), S4_FAST(weight_grads),
                           S4_FAST(swiglu), S4_FAST(swiglu_backward),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_act8", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__act8() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "built_for", ACT8_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
