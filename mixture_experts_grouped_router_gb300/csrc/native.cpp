// Python calls of the short low-bit operators: the tensors' pointers, sizes and
// leading dimensions are taken here and handed to the C ABI.  A call's kernels take a
// few microseconds, so that the host's share counts: 3.2 us a call on an Arm core
// with the launch (1.5), where ctypes takes 5.5.  `_lib.py` holds the functions
// that a program calls, with their words, and raises what these return.
//
// Every function takes its arguments by position, tensors as such (None where the C
// ABI takes a null pointer), the stream as an integer last, and returns the status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "moe_gb300.h"

namespace {

PyObject *s_data_ptr, *s_stride, *s_numel, *s_shape;

// An argument's value, or an error that ends the call.
struct Failed {};

int64_t as_int(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  return v;
}

int as_int32(int64_t v) {
  if (v != (int)v) {
    PyErr_Format(PyExc_OverflowError, "%lld does not fit 32 bits", (long long)v);
    throw Failed{};
  }
  return (int)v;
}

int int32_arg(PyObject *o) { return as_int32(as_int(o)); }

int64_t call_int(PyObject *t, PyObject *name) {
  PyObject *r = PyObject_CallMethodNoArgs(t, name);
  if (r == nullptr) throw Failed{};
  const unsigned long long v = PyLong_AsUnsignedLongLong(r);
  Py_DECREF(r);
  if (v == (unsigned long long)-1 && PyErr_Occurred()) throw Failed{};
  return (int64_t)v;
}

// Element i of a tuple of integers, from the end where i < 0.
int64_t item(PyObject *tuple, Py_ssize_t i) {
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  if (i < 0) i += n;
  if (i < 0 || i >= n) {
    PyErr_SetString(PyExc_IndexError, "a tensor of too few dimensions");
    throw Failed{};
  }
  return as_int(PyTuple_GET_ITEM(tuple, i));
}

// A tuple that goes with the scope.
struct Tuple {
  PyObject *o;
  explicit Tuple(PyObject *p) : o(p) {
    if (o != nullptr && !PyTuple_Check(o)) {
      Py_DECREF(o);
      o = nullptr;
      PyErr_SetString(PyExc_TypeError, "a tensor's shape and strides are tuples");
    }
    if (o == nullptr) throw Failed{};
  }
  ~Tuple() { Py_XDECREF(o); }
  Tuple(const Tuple &) = delete;
};

int64_t dim(PyObject *t, Py_ssize_t i) {
  Tuple s(PyObject_GetAttr(t, s_shape));
  return item(s.o, i);
}

// rows and columns of a matrix
void sizes(PyObject *t, int64_t &rows, int &cols) {
  Tuple s(PyObject_GetAttr(t, s_shape));
  if (PyTuple_GET_SIZE(s.o) != 2) {
    PyErr_SetString(PyExc_ValueError, "matrices only");
    throw Failed{};
  }
  rows = item(s.o, 0);
  cols = as_int32(item(s.o, 1));
}

template <typename T>
T *ptr(PyObject *t) {
  return t == Py_None ? nullptr : reinterpret_cast<T *>(call_int(t, s_data_ptr));
}

int64_t numel(PyObject *t) { return t == Py_None ? 0 : call_int(t, s_numel); }

// The leading dimension of a row-major matrix.
int64_t ld(PyObject *t) {
  Tuple s(PyObject_CallMethodNoArgs(t, s_stride));
  if (PyTuple_GET_SIZE(s.o) < 2) {
    PyErr_SetString(PyExc_AssertionError, "matrices only");
    throw Failed{};
  }
  const bool empty = call_int(t, s_numel) == 0;
  if (empty) return dim(t, -1);
  if (item(s.o, -1) != 1) {
    PyErr_SetString(PyExc_AssertionError, "row-major tensors only");
    throw Failed{};
  }
  return item(s.o, -2);
}

// group_offsets and the number of groups that it bounds
const int32_t *offsets(PyObject *t, int &E, int without) {
  E = without;
  if (t == Py_None) return nullptr;
  E = as_int32(dim(t, 0) - 1);
  return ptr<int32_t>(t);
}

moe_stream_t stream(PyObject *o) { return reinterpret_cast<moe_stream_t>(as_int(o)); }

// Runs `f` on the arguments without the interpreter's lock around the C call.
template <int N, typename F>
PyObject *entry(PyObject *const *a, Py_ssize_t n, F f) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f(a));
  } catch (const Failed &) {
    return nullptr;
  }
}

template <typename F>
moe_status_t unlocked(F f) {
  moe_status_t st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// x, q, scales, group_offsets, stream
PyObject *act8_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<5>(args, n, [](PyObject *const *a) {
    int64_t rows;
    int cols, E;
    sizes(a[0], rows, cols);
    const int32_t *off = offsets(a[3], E, 0);
    const auto x = ptr<uint16_t>(a[0]);
    const auto q = ptr<int8_t>(a[1]);
    const auto s = ptr<uint16_t>(a[2]);
    const int64_t ldx = ld(a[0]), ldq = ld(a[1]), lds = ld(a[2]);
    const moe_stream_t st = stream(a[4]);
    return unlocked([=] { return moe_act8_quantize(x, ldx, rows, cols, off, E, q, ldq, s, lds, st); });
  });
}

// q, scales, x, group_offsets, stream
PyObject *act8_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<5>(args, n, [](PyObject *const *a) {
    int64_t rows;
    int cols, E;
    sizes(a[2], rows, cols);
    const int32_t *off = offsets(a[3], E, 0);
    const auto q = ptr<int8_t>(a[0]);
    const auto s = ptr<uint16_t>(a[1]);
    const auto x = ptr<uint16_t>(a[2]);
    const int64_t ldq = ld(a[0]), lds = ld(a[1]), ldx = ld(a[2]);
    const moe_stream_t st = stream(a[4]);
    return unlocked([=] { return moe_act8_dequantize(q, ldq, s, lds, rows, cols, off, E, x, ldx, st); });
  });
}

// h, act, q, scales, group_offsets, stream
PyObject *act8_swiglu_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject *const *a) {
    int64_t rows;
    int F, E;
    sizes(a[1], rows, F);
    const int32_t *off = offsets(a[4], E, 0);
    const auto h = ptr<uint16_t>(a[0]);
    const auto act = ptr<uint16_t>(a[1]);
    const auto q = ptr<int8_t>(a[2]);
    const auto s = ptr<uint16_t>(a[3]);
    const int64_t ldh = ld(a[0]), lda = ld(a[1]), ldq = ld(a[2]), lds = ld(a[3]);
    const moe_stream_t st = stream(a[5]);
    return unlocked([=] {
      return moe_act8_swiglu_fwd(h, ldh, rows, F, off, E, act, lda, q, ldq, s, lds, st);
    });
  });
}

// q, scales, dact, dh, act, group_offsets, stream
PyObject *act8_swiglu_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<7>(args, n, [](PyObject *const *a) {
    int64_t rows;
    int F, E;
    sizes(a[2], rows, F);
    const int32_t *off = offsets(a[5], E, 0);
    const auto q = ptr<int8_t>(a[0]);
    const auto s = ptr<uint16_t>(a[1]);
    const auto dact = ptr<uint16_t>(a[2]);
    const auto dh = ptr<uint16_t>(a[3]);
    const auto act = ptr<uint16_t>(a[4]);
    const int64_t ldq = ld(a[0]), lds = ld(a[1]), ldd = ld(a[2]), ldh = ld(a[3]);
    const int64_t lda = a[4] == Py_None ? 0 : ld(a[4]);
    const moe_stream_t st = stream(a[6]);
    return unlocked([=] {
      return moe_act8_swiglu_bwd(q, ldq, s, lds, dact, ldd, rows, F, off, E, dh, ldh, act, lda, st);
    });
  });
}

// x, fmt, q, sf, row_map, group_offsets, groups, row_index, index_div, scale, workspace,
// dev_status, stream
PyObject *fp4_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<13>(args, n, [](PyObject *const *a) {
    int64_t src_rows;
    int cols, E;
    sizes(a[0], src_rows, cols);
    const int fmt = int32_arg(a[1]), map = int32_arg(a[4]);
    const int32_t *off = offsets(a[5], E, int32_arg(a[6]));
    const int64_t rows = dim(a[2], 0);
    const auto x = ptr<uint16_t>(a[0]);
    const auto q = ptr<uint8_t>(a[2]);
    const auto sf = ptr<uint8_t>(a[3]);
    const auto index = ptr<int32_t>(a[7]);
    const int div = int32_arg(a[8]);
    const auto scale = ptr<float>(a[9]);
    void *const ws = ptr<void>(a[10]);
    const auto status = ptr<int32_t>(a[11]);
    const int64_t ldx = ld(a[0]), ldq = ld(a[2]);
    const size_t sf_bytes = numel(a[3]), ws_bytes = numel(a[10]);
    const moe_stream_t st = stream(a[12]);
    return unlocked([=] {
      return moe_fp4_quantize(x, ldx, src_rows, index, div, rows, cols, fmt, map, off, E, scale, q,
                              ldq, sf, sf_bytes, ws, ws_bytes, status, st);
    });
  });
}

// q, sf, fmt, x, row_map, group_offsets, groups, scale, stream
PyObject *fp4_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<9>(args, n, [](PyObject *const *a) {
    int64_t rows;
    int cols, E;
    sizes(a[3], rows, cols);
    const int fmt = int32_arg(a[2]), map = int32_arg(a[4]);
    const int32_t *off = offsets(a[5], E, int32_arg(a[6]));
    const auto q = ptr<uint8_t>(a[0]);
    const auto sf = ptr<uint8_t>(a[1]);
    const auto x = ptr<uint16_t>(a[3]);
    const auto scale = ptr<float>(a[7]);
    const int64_t ldq = ld(a[0]), ldx = ld(a[3]);
    const size_t sf_bytes = numel(a[1]);
    const moe_stream_t st = stream(a[8]);
    return unlocked([=] {
      return moe_fp4_dequantize(q, ldq, sf, sf_bytes, rows, cols, fmt, map, off, E, scale, x, ldx, st);
    });
  });
}

// addresses of moe_fp4_weights and moe_fp4_buffers, x, sorted_to_flat, k, group_offsets, stream
PyObject *fp4_experts(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<7>(args, n, [](PyObject *const *a) {
    const auto w = reinterpret_cast<const moe_fp4_weights *>(as_int(a[0]));
    const auto b = reinterpret_cast<const moe_fp4_buffers *>(as_int(a[1]));
    int64_t T;
    int d;
    sizes(a[2], T, d);
    const int tokens = as_int32(T), k = int32_arg(a[4]);
    const auto x = ptr<uint16_t>(a[2]);
    const auto s2f = ptr<int32_t>(a[3]);
    const auto off = ptr<int32_t>(a[5]);
    const int64_t ldx = ld(a[2]);
    const moe_stream_t st = stream(a[6]);
    return unlocked([=] { return moe_fp4_experts(w, b, x, ldx, tokens, s2f, k, off, st); });
  });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"act8_quantize", fast(act8_quantize), METH_FASTCALL, nullptr},
    {"act8_dequantize", fast(act8_dequantize), METH_FASTCALL, nullptr},
    {"act8_swiglu_fwd", fast(act8_swiglu_fwd), METH_FASTCALL, nullptr},
    {"act8_swiglu_bwd", fast(act8_swiglu_bwd), METH_FASTCALL, nullptr},
    {"fp4_quantize", fast(fp4_quantize), METH_FASTCALL, nullptr},
    {"fp4_dequantize", fast(fp4_dequantize), METH_FASTCALL, nullptr},
    {"fp4_experts", fast(fp4_experts), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) {
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_numel = PyUnicode_InternFromString("numel");
  s_shape = PyUnicode_InternFromString("shape");
  if (s_data_ptr == nullptr || s_stride == nullptr || s_numel == nullptr || s_shape == nullptr)
    return nullptr;
  return PyModule_Create(&module);
}
