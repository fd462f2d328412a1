// Argument marshalling of libpa's calls for Python: torch tensors to pa_tensor descriptors, the
// current stream, one C call.  Built as the extension module _marshal; the functions of libpa come
// to it as addresses (bind), so that one copy of the library serves both this module and ctypes.
//
// A descriptor made in Python costs about a microsecond, and these calls take up to nine
// tensors: more time than a decode step's kernels need.  Here a whole call takes about one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cstring>
#include <exception>

#include "pa.h"

namespace {

decltype(&pa_cache_append_rope) g_append_rope;
decltype(&pa_cache_append_q4) g_append_q4;
decltype(&pa_cache_read_q4) g_read_q4;
decltype(&pa_decode_q4) g_decode_q4;
decltype(&pa_block_bounds) g_block_bounds;
decltype(&pa_select_blocks) g_select_blocks;
decltype(&pa_decode_selected) g_decode_selected;

struct Function {
  const char* name;
  void* at;
};
Function g_functions[] = {
    {"pa_cache_append_rope", &g_append_rope}, {"pa_cache_append_q4", &g_append_q4},
    {"pa_cache_read_q4", &g_read_q4},         {"pa_decode_q4", &g_decode_q4},
    {"pa_block_bounds", &g_block_bounds},     {"pa_select_blocks", &g_select_blocks},
    {"pa_decode_selected", &g_decode_selected},
};

// One call's arguments.  Every method returns false with a Python exception set.
struct Call {
  static constexpr int kMost = 9;
  pa_tensor desc[kMost];
  int used = 0;
  int device = -1;

  // *out = descriptor of a CUDA tensor on the current device; None: NULL, where `optional`
  bool tensor(PyObject* o, const pa_tensor** out, bool optional = false) {
    *out = nullptr;
    if (optional && o == Py_None) return true;
    if (!THPVariable_Check(o)) {
      PyErr_Format(PyExc_TypeError, "expected a tensor, got %.100s", Py_TYPE(o)->tp_name);
      return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) {
      PyErr_SetString(PyExc_ValueError, "device operations take CUDA tensors");
      return false;
    }
    if (device < 0) device = c10::cuda::current_device();
    if (t.get_device() != device) {
      PyErr_Format(PyExc_ValueError, "tensor on cuda:%d but the current device is cuda:%d", static_cast<int>(t.get_device()),
                   device);
      return false;
    }
    pa_tensor& d = desc[used++];
    switch (t.scalar_type()) {
      case at::kFloat: d.dtype = PA_F32; break;
      case at::kHalf: d.dtype = PA_F16; break;
      case at::kBFloat16: d.dtype = PA_BF16; break;
      case at::kInt: d.dtype = PA_I32; break;
      case at::kByte: d.dtype = PA_U8; break;
      default: PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type())); return false;
    }
    if (t.dim() < 1 || t.dim() > 4) {
      PyErr_SetString(PyExc_ValueError, "tensors must have 1..4 dims");
      return false;
    }
    d.ndim = static_cast<int32_t>(t.dim());
    for (int i = 0; i < d.ndim; ++i) {
      d.shape[i] = t.size(i);
      d.stride[i] = t.stride(i);
    }
    d.data = t.numel() ? t.data_ptr() : nullptr;
    *out = &d;
    return true;
  }

  bool number(PyObject* o, int32_t* out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if (v < INT32_MIN || v > INT32_MAX) {
      PyErr_SetString(PyExc_OverflowError, "integer argument outside int32");
      return false;
    }
    *out = static_cast<int32_t>(v);
    return true;
  }

  bool real(PyObject* o, float* out) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    *out = static_cast<float>(v);
    return true;
  }

  // a torch.cuda.Stream, or None: the device's current stream
  bool stream(PyObject* o, pa_stream* out) {
    if (o == Py_None) {
      *out = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
      return true;
    }
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) return false;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
  }
};

bool count_is(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// Runs f without the interpreter lock; its return code as an int.
template <typename F>
PyObject* run(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

// No C++ exception crosses into the interpreter.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <typename Fn>
PyObject* append(Fn fn, PyObject* const* a, Py_ssize_t n) {
  // k_new, v_new, slots, k_cache, v_cache, positions, cos_sin, interleaved, q, q_out, stream
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor* t[9];
    int32_t inter;
    pa_stream st;
    if (!count_is(n, 11)) return nullptr;
    for (int i = 0; i < 7; ++i)
      if (!c.tensor(a[i], &t[i], i >= 5)) return nullptr;
    if (!c.number(a[7], &inter) || !c.tensor(a[8], &t[7], true) || !c.tensor(a[9], &t[8], true) || !c.stream(a[10], &st))
      return nullptr;
    return run([&] { return fn(t[0], t[1], t[2], t[3], t[4], t[5], t[6], inter, t[7], t[8], st); });
  });
}

PyObject* py_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) { return append(g_append_rope, a, n); }
PyObject* py_append_q4(PyObject*, PyObject* const* a, Py_ssize_t n) { return append(g_append_q4, a, n); }

PyObject* py_read_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor* t[5];
    pa_stream st;
    if (!count_is(n, 6)) return nullptr;
    for (int i = 0; i < 5; ++i)
      if (!c.tensor(a[i], &t[i])) return nullptr;
    if (!c.stream(a[5], &st)) return nullptr;
    return run([&] { return g_read_q4(t[0], t[1], t[2], t[3], t[4], st); });
  });
}

PyObject* py_decode_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // q, k_cache, v_cache, block_tables, context_lens, scale, out, stream
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor *t[5], *out;
    float scale;
    pa_stream st;
    if (!count_is(n, 8)) return nullptr;
    for (int i = 0; i < 5; ++i)
      if (!c.tensor(a[i], &t[i])) return nullptr;
    if (!c.real(a[5], &scale) || !c.tensor(a[6], &out) || !c.stream(a[7], &st)) return nullptr;
    return run([&] { return g_decode_q4(t[0], t[1], t[2], t[3], t[4], scale, out, st); });
  });
}

PyObject* py_block_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // k_cache, block_tables, context_lens, first_tokens, bounds, stream
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor* t[5];
    pa_stream st;
    if (!count_is(n, 6)) return nullptr;
    for (int i = 0; i < 5; ++i)
      if (!c.tensor(a[i], &t[i], i == 3)) return nullptr;
    if (!c.stream(a[5], &st)) return nullptr;
    return run([&] { return g_block_bounds(t[0], t[1], t[2], t[3], t[4], st); });
  });
}

PyObject* py_select_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // q, bounds, block_tables, context_lens, block_size, keep_first, keep_last, selected, stream
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor *t[4], *sel;
    int32_t v[3];
    pa_stream st;
    if (!count_is(n, 9)) return nullptr;
    for (int i = 0; i < 4; ++i)
      if (!c.tensor(a[i], &t[i])) return nullptr;
    for (int i = 0; i < 3; ++i)
      if (!c.number(a[4 + i], &v[i])) return nullptr;
    if (!c.tensor(a[7], &sel) || !c.stream(a[8], &st)) return nullptr;
    return run([&] { return g_select_blocks(t[0], t[1], t[2], t[3], v[0], v[1], v[2], sel, st); });
  });
}

PyObject* py_decode_selected(PyObject*, PyObject* const* a, Py_ssize_t n) {
  // q, k_cache, v_cache, block_tables, context_lens, selected, scale, out, stream
  return guarded([&]() -> PyObject* {
    Call c;
    const pa_tensor *t[6], *out;
    float scale;
    pa_stream st;
    if (!count_is(n, 9)) return nullptr;
    for (int i = 0; i < 6; ++i)
      if (!c.tensor(a[i], &t[i])) return nullptr;
    if (!c.real(a[6], &scale) || !c.tensor(a[7], &out) || !c.stream(a[8], &st)) return nullptr;
    return run([&] { return g_decode_selected(t[0], t[1], t[2], t[3], t[4], t[5], scale, out, st); });
  });
}

// bind(name, address): where a function of libpa is
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count_is(n, 2)) return nullptr;
  const char* name = PyUnicode_AsUTF8(a[0]);
  if (!name) return nullptr;
  void* p = PyLong_AsVoidPtr(a[1]);
  if (PyErr_Occurred()) return nullptr;
  for (Function& f : g_functions)
    if (std::strcmp(f.name, name) == 0) {
      std::memcpy(f.at, &p, sizeof(p));
      Py_RETURN_NONE;
    }
  PyErr_Format(PyExc_KeyError, "%s", name);
  return nullptr;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef g_methods[] = {
    {"bind", FAST(py_bind)},
    {"pa_cache_append_rope", FAST(py_append_rope)},
    {"pa_cache_append_q4", FAST(py_append_q4)},
    {"pa_cache_read_q4", FAST(py_read_q4)},
    {"pa_decode_q4", FAST(py_decode_q4)},
    {"pa_block_bounds", FAST(py_block_bounds)},
    {"pa_select_blocks", FAST(py_select_blocks)},
    {"pa_decode_selected", FAST(py_decode_selected)},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
  PyObject* m = PyModule_Create(&g_module);
  // the torch whose tensor layout this file was compiled for
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
