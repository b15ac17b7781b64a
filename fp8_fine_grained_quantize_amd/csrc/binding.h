// What the parts of the Python binding share: checks of arguments, outputs, the
// interpreter's lock, and the wrapper that turns C++ exceptions into Python's.
#pragma once

#include <ATen/ops/empty.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/python_headers.h>

#include <initializer_list>
#include <string>
#include <utility>

#include "../../include/libfp8blk.h"

namespace fp8blk_py {

using at::Tensor;
using c10::ScalarType;

// An argument that is refused: the Python exception to raise.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] inline void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] inline void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

inline std::string sizes(const Tensor& t) {
  std::string s = "(";
  for (int64_t n : t.sizes()) s += std::to_string(n) + ",";
  return s + ")";
}

inline const Tensor* maybe(PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
inline const Tensor& given(PyObject* o, const char* what) {
  const Tensor* t = maybe(o, what);
  if (t == nullptr) type_error(std::string(what) + " must be a tensor");
  return *t;
}
inline int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
inline double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
inline bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

inline void* addr(const Tensor* t) { return t == nullptr ? nullptr : const_cast<void*>(t->const_data_ptr()); }
inline void* addr(const Tensor& t) { return addr(&t); }

inline void need(const Tensor& t, ScalarType dtype, const char* what) {
  if (t.scalar_type() != dtype)
    type_error(std::string(what) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
}
inline bool is_f32(const Tensor& t, const char* what) {
  if (t.scalar_type() == at::kFloat) return true;
  if (t.scalar_type() == at::kBFloat16) return false;
  type_error(std::string(what) + " must be float32 or bfloat16, got " + c10::toString(t.scalar_type()));
}
inline void matrix(const Tensor& t, int64_t rows, int64_t cols, const char* what) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    value_error(std::string(what) + " must have shape (" + std::to_string(rows) + "," + std::to_string(cols) + "), got " +
                sizes(t));
}
inline void two_d(const Tensor& t, const char* what) {
  if (t.dim() != 2) value_error(std::string(what) + " must be a matrix, got shape " + sizes(t));
}

// Row pitch of a row-major matrix, in elements.
inline int64_t pitch(const Tensor& t, const char* what) {
  const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0), step = t.stride(1);
  if (rows == 0 || cols == 0) {
    const int64_t per = 16 / t.element_size();
    return (cols + per - 1) / per * per;
  }
  if ((step != 1 && cols != 1) || (ld < cols && rows != 1))
    value_error(std::string(what) + " must be a row-major matrix of separate rows, got strides (" + std::to_string(ld) +
                "," + std::to_string(step) + ")");
  return ld >= cols ? ld : cols;
}
inline int64_t pitch(const Tensor& t, ScalarType dtype, int64_t rows, int64_t cols, const char* what) {
  need(t, dtype, what);
  matrix(t, rows, cols, what);
  return pitch(t, what);
}

inline void dense(const Tensor& t, ScalarType dtype, std::initializer_list<int64_t> shape, const char* what) {
  need(t, dtype, what);
  if (t.sizes() != c10::IntArrayRef(shape)) value_error(std::string(what) + " has the wrong shape: " + sizes(t));
  if (!t.is_contiguous()) value_error(std::string(what) + " must be contiguous");
}

// Memory the caller lends a call: its bytes are counted from its size.
inline void scratch(const Tensor* t) {
  if (t != nullptr && !t->is_contiguous()) value_error("workspace must be contiguous");
}

// The interpreter's lock, given up while outputs are allocated and the launch
// is queued: both can wait for the device.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  void end() {
    if (state != nullptr) PyEval_RestoreThread(state);
    state = nullptr;
  }
  ~Unlocked() { end(); }
};

// The stream's handle, once every tensor is known to lie on the first one's device.
inline void* stream_of(PyObject* stream, const Tensor& first, std::initializer_list<const Tensor*> others) {
  if (stream == Py_None) value_error("expected tensors on the current GPU, got " + first.device().str());
  for (const Tensor* t : others)
    if (t != nullptr && t->device() != first.device())
      value_error("tensors on different devices: " + first.device().str() + " and " + t->device().str());
  return reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(stream)));
}

// Outputs and workspaces that the caller lends, before their addresses are
// taken: one that shares its memory with a tensor until either is written (a
// copy-on-write clone) gets its own here.  Inputs are read where they are.
inline void own(std::initializer_list<const Tensor*> lent) {
  for (const Tensor* t : lent)
    if (t != nullptr) t->mutable_data_ptr();
}

// A kernel wrote this tensor of the caller's: autograd refuses a graph that still
// needs the old values, as after torch's own in-place operations.  (Tensors of
// inference mode have no versions.)
inline void wrote(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
inline void wrote(std::initializer_list<const Tensor*> lent) {
  for (const Tensor* t : lent)
    if (t != nullptr) wrote(*t);
}

inline Tensor vec(std::initializer_list<int64_t> shape, ScalarType dtype, const Tensor& like) {
  return at::empty(c10::IntArrayRef(shape), at::TensorOptions().dtype(dtype).device(like.device()));
}

// The given output, checked, or a new matrix whose rows lie a multiple of 16
// bytes apart; `ld` receives the pitch.
inline Tensor output(const Tensor* t, int64_t rows, int64_t cols, ScalarType dtype, const Tensor& like, const char* what,
              int64_t& ld) {
  if (t != nullptr) {
    ld = pitch(*t, dtype, rows, cols, what);
    return *t;
  }
  const int64_t per = 16 / static_cast<int64_t>(c10::elementSize(dtype));
  ld = (cols + per - 1) / per * per;
  Tensor n = vec({rows, ld}, dtype, like);
  return ld == cols ? n : n.narrow(1, 0, cols);
}

inline PyObject* g_error = nullptr;  // Fp8BlkError

inline void ok(fp8blk_status_t status, const char* what) {
  if (status != FP8BLK_OK)
    throw Refused{g_error != nullptr ? g_error : PyExc_RuntimeError,
                  std::string(what) + " failed: " + fp8blk_status_string(status)};
}

inline PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
// A tensor for Python, None for an undefined one.
inline PyObject* wrap_maybe(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
inline PyObject* tuple(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) PyTuple_SET_ITEM(r, i++, wrap_maybe(*t));
  return r;
}

inline ScalarType dtype_of(PyObject* o) {
  if (!THPDtype_Check(o)) type_error("expected a torch.dtype");
  const ScalarType d = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (d != at::kFloat && d != at::kBFloat16)
    type_error(std::string("output type must be float32 or bfloat16, got ") + c10::toString(d));
  return d;
}

// Rows of `width` bytes, `pitch` (at least the width) apart.
struct Span {
  int64_t base, width, pitch, rows;
  int64_t end() const { return base + (rows - 1) * pitch + width; }
};

// Whether two spans have a byte in common, exactly: rows may lie between rows.
inline bool meet(Span a, Span b) {
  if (a.rows > b.rows) std::swap(a, b);
  if (a.pitch == b.pitch && a.rows > 1) {  // only the distance of the rows counts: one row against all of them
    b.base -= (a.rows - 1) * a.pitch;
    b.rows += a.rows - 1;
    a.rows = 1;
  }
  for (int64_t i = 0; i < a.rows; ++i) {
    const int64_t lo = a.base + i * a.pitch, past = lo - b.width - b.base;  // b's rows up to `past` end before lo
    const int64_t j = past < 0 ? 0 : past / b.pitch + 1;
    if (j < b.rows && b.base + j * b.pitch < lo + a.width) return true;
  }
  return false;
}

// No C++ exception leaves the module: refusals and torch's own become Python's.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

}  // namespace fp8blk_py

#define FP8BLK_METHOD(NAME, N) \
  {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&fp8blk_py::call<NAME, N>)), METH_FASTCALL, nullptr}
