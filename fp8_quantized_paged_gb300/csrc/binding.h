// binding.h -- what the Python bindings of libkvq share: arguments by position or
// name, the checks that the C ABI cannot make from a pointer, errors.
#pragma once

#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cstdio>
#include <string>

#include "../../include/kvq.h"

namespace binding {

constexpr int kBlockSize = 16;

extern PyObject* g_error;  // KvqError(status, text)

// Thrown once a Python error is set.
struct Raised {};

[[noreturn]] inline void fail(const char* where, const std::string& text, int status) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, (std::string(where) + ": " + text).c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// One call's arguments by position: positional first, then by name; absent
// ones stay NULL.  `need` of the names have to be there.
template <size_t N>
std::array<PyObject*, N> take(const char* where, const char* const (&names)[N], size_t need,
                              PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  std::array<PyObject*, N> got{};
  if (static_cast<size_t>(nargs) > N) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %zu arguments (%zd given)", where, N, nargs);
    throw Raised();
  }
  for (Py_ssize_t i = 0; i < nargs; ++i) got[i] = args[i];
  const Py_ssize_t nkw = kw ? PyTuple_GET_SIZE(kw) : 0;
  for (Py_ssize_t i = 0; i < nkw; ++i) {
    PyObject* name = PyTuple_GET_ITEM(kw, i);
    size_t k = 0;
    while (k < N && PyUnicode_CompareWithASCIIString(name, names[k]) != 0) ++k;
    if (k == N || got[k]) {
      PyErr_Format(PyExc_TypeError, "%s() got %s argument '%U'", where,
                   k == N ? "an unexpected" : "twice the", name);
      throw Raised();
    }
    got[k] = args[nargs + i];
  }
  for (size_t k = 0; k < need; ++k)
    if (!got[k]) {
      PyErr_Format(PyExc_TypeError, "%s() misses the argument '%s'", where, names[k]);
      throw Raised();
    }
  return got;
}

inline long long integer(const char* where, const char* name, PyObject* o, long long most) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    fail(where, std::string(name) + " must be an integer", KVQ_ERR_ARG);
  }
  // (values past the C type would wrap; the library refuses what is below 0)
  if (v > most || v < -most) fail(where, std::string(name) + " is out of range", KVQ_ERR_ARG);
  return v;
}

inline int int32(const char* where, const char* name, PyObject* o) {
  return static_cast<int>(integer(where, name, o, 0x7FFFFFFFll));
}

inline std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// The tensors of one call, and where they are.
class Tensors {
 public:
  explicit Tensors(const char* where) : where_(where) {}

  const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "%s: %s must be a tensor", where_, name);
      throw Raised();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    const c10::Device d = t.device();
    const int at = d.is_cuda() ? d.index() : -1;
    if (count_++ == 0) {
      device_ = at;
      first_ = name;
    } else if (at != device_ && !other_) {
      other_ = name;
    }
    return t;
  }

  // A dense tensor of this type.
  void* dense(const char* name, const at::Tensor& t, c10::ScalarType type) {
    if (t.scalar_type() != type)
      fail(where_, std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()), KVQ_ERR_ARG);
    if (!t.is_contiguous()) fail(where_, std::string(name) + " must be contiguous", KVQ_ERR_SHAPE);
    return t.data_ptr();
  }
  void* dense(const char* name, PyObject* o, c10::ScalarType type, int64_t* numel = nullptr) {
    const at::Tensor& t = tensor(name, o);
    if (numel) *numel = t.numel();
    return dense(name, t, type);
  }
  void* dense(const char* name, PyObject* o, c10::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(name, o);
    void* p = dense(name, t, type);
    if (t.sizes() != shape)
      fail(where_, std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()), KVQ_ERR_SHAPE);
    return p;
  }

  // bf16 rows [n][heads][head_dim], dense but for the distance of consecutive rows.
  void* rows(const char* name, const at::Tensor& t, int64_t n, int64_t heads, int64_t dh, int64_t& distance) {
    if (t.scalar_type() != at::kBFloat16)
      fail(where_, std::string(name) + " must be " + c10::toString(at::kBFloat16) + ", got " + c10::toString(t.scalar_type()), KVQ_ERR_ARG);
    const int64_t want[3] = {n, heads, dh};
    if (t.sizes() != at::IntArrayRef(want, 3))
      fail(where_, std::string(name) + " must have shape " + shape_text(at::IntArrayRef(want, 3)) + ", got " + shape_text(t.sizes()), KVQ_ERR_SHAPE);
    if ((heads > 1 && t.stride(1) != dh) || t.stride(2) != 1)
      fail(where_, std::string(name) + " must be dense within a row", KVQ_ERR_SHAPE);
    distance = n > 1 ? t.stride(0) : heads * dh;
    return t.data_ptr();
  }

  uint32_t* status(PyObject* o) {
    if (!o || o == Py_None) return nullptr;
    const at::Tensor& t = tensor("dev_status", o);
    if (t.element_size() != 4 || t.numel() < 1) fail(where_, "dev_status must hold a 32-bit word", KVQ_ERR_ARG);
    return static_cast<uint32_t*>(t.data_ptr());
  }

  // After the other checks: all tensors on CUDA's current device, where the kernels
  // run; and the call's stream (None: the current one; a stream, or its address).
  kvq_stream_t stream(PyObject* o) {
    if (device_ < 0) fail(where_, std::string(first_) + " must be a CUDA tensor", KVQ_ERR_ARG);
    if (other_) fail(where_, std::string(other_) + " must be on the device of " + first_, KVQ_ERR_ARG);
    if (device_ != c10::cuda::current_device())
      fail(where_, std::string(first_) + " must be on the current device", KVQ_ERR_ARG);
    if (!o || o == Py_None)
      return reinterpret_cast<kvq_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream());
    PyObject* a = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!a) throw Raised();
    void* p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    if (PyErr_Occurred()) throw Raised();
    return reinterpret_cast<kvq_stream_t>(p);
  }

 private:
  const char* where_;
  int count_ = 0, device_ = -1;
  const char* first_ = "";
  const char* other_ = nullptr;
};

inline int narrow(const char* where, const char* what, int64_t v) {
  if (v > 0x7FFFFFFF) fail(where, std::string("too many ") + what, KVQ_ERR_UNSUPPORTED);
  return static_cast<int>(v);
}

inline PyObject* result(const char* where, int status) {
  if (status != KVQ_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  Py_RETURN_NONE;
}

// Runs f with Python's errors and C++'s kept apart from each other.
template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The entry points of kvq_step.h in the library `handle` (false, with a Python error set, where one is
// missing), and their methods, the last of them empty.
bool step_bind(void* handle, const char* path);
extern PyMethodDef step_methods[];

}  // namespace binding
