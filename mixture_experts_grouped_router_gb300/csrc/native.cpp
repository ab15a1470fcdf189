// Python calls of the short operators (low-bit formats, and what a step has around the
// expert layer): the tensors' pointers, sizes and
// leading dimensions are taken here and handed to the C ABI.  A call's kernels take a
// few microseconds, so that the host's share counts: 3.2 us a call on an Arm core
// with the launch (1.5), where ctypes takes 5.5.  `_lib.py` holds the functions
// that a program calls, with their words, and raises what these return.
//
// Every function takes its arguments by position, tensors as such (None where the C
// ABI takes a null pointer), the stream as an integer last, and returns the status.
// The C ABI knows addresses and leading dimensions alone; that every operand has the
// rows, columns and elements which the call's sizes name, and their type, is checked here
// (ValueError).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <initializer_list>

#include "moe_gb300.h"

namespace {

PyObject *t_bf16, *t_u8, *t_i8, *t_i32, *t_f32;  // torch's types

// A method or an attribute of a tensor, by its descriptor in torch's tensor type (which
// saves the look-up); of what is no tensor by its name, which fails as in Python.
PyTypeObject *tensor_type;
struct Member {
  const char *text;
  PyObject *name, *descr;
  PyObject *call(PyObject *t) const {
    if (!PyObject_TypeCheck(t, tensor_type)) return PyObject_CallMethodNoArgs(t, name);
    return PyObject_Vectorcall(descr, &t, 1, nullptr);
  }
  PyObject *get(PyObject *t) const {
    if (!PyObject_TypeCheck(t, tensor_type)) return PyObject_GetAttr(t, name);
    return Py_TYPE(descr)->tp_descr_get(descr, t, (PyObject *)Py_TYPE(t));
  }
};
Member m_data_ptr = {"data_ptr"}, m_stride = {"stride"}, m_numel = {"numel"}, m_shape = {"shape"},
       m_is_contiguous = {"is_contiguous"}, m_dtype = {"dtype"}, m_get_device = {"get_device"};

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

int64_t call_int(PyObject *t, const Member &m) {
  PyObject *r = m.call(t);
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

bool is_contiguous(PyObject *t) {
  PyObject *r = m_is_contiguous.call(t);
  if (r == nullptr) throw Failed{};
  Py_DECREF(r);
  return r == Py_True;
}

// `name` of the call holds elements of `type`; any type of one byte where that is uint8
// (codes and scales, as which of them they are called).
void check_type(const char *name, PyObject *t, PyObject *type) {
  PyObject *d = m_dtype.get(t);
  if (d == nullptr) throw Failed{};
  bool ok = d == type || (d == t_i8 && type == t_u8);
  if (!ok && type == t_u8) {
    PyObject *size = PyObject_GetAttrString(d, "itemsize");
    ok = size != nullptr && PyLong_AsLong(size) == 1;
    Py_XDECREF(size);
    PyErr_Clear();
  }
  if (!ok) PyErr_Format(PyExc_ValueError, "%s is %S, not %S", name, d, type);
  Py_DECREF(d);
  if (!ok) throw Failed{};
}

// A row-major matrix (the last two dimensions of a tensor).
struct Matrix {
  void *p;
  int64_t rows, cols, ld;
  template <typename T>
  T *as() const {
    return static_cast<T *>(p);
  }
};

Matrix matrix(const char *name, PyObject *t, PyObject *type, bool exact = false) {
  Tuple shape(m_shape.get(t));
  const Py_ssize_t dims = PyTuple_GET_SIZE(shape.o);
  if (dims < 2 || (exact && dims > 2)) {
    PyErr_SetString(exact ? PyExc_ValueError : PyExc_AssertionError, "matrices only");
    throw Failed{};
  }
  Matrix m;
  m.rows = item(shape.o, -2);
  m.cols = m.ld = item(shape.o, -1);
  if (!is_contiguous(t)) {  // (neither an empty one nor a single row is)
    Tuple stride(m_stride.call(t));
    if (item(stride.o, -1) != 1) {
      PyErr_SetString(PyExc_AssertionError, "row-major tensors only");
      throw Failed{};
    }
    m.ld = item(stride.o, -2);
  }
  check_type(name, t, type);
  m.p = reinterpret_cast<void *>(call_int(t, m_data_ptr));
  return m;
}

// m, `name` of the call, has to hold `rows` rows of `cols` columns.  A leading dimension
// under that is left to the library, which refuses it.
void need(const char *name, const Matrix &m, int64_t rows, int64_t cols) {
  if (rows <= 0 || (m.rows >= rows && (m.cols >= cols || m.ld < cols))) return;
  PyErr_Format(PyExc_ValueError, "%s is [%lld, %lld] for [%lld, %lld]", name, (long long)m.rows,
               (long long)m.cols, (long long)rows, (long long)cols);
  throw Failed{};
}

// The elements of a contiguous tensor; none of None (an empty tensor has no address either).
struct Vector {
  void *p = nullptr;
  int64_t n = 0;
  bool given = false;
  template <typename T>
  T *as() const {
    return static_cast<T *>(p);
  }
};

Vector vector(const char *name, PyObject *t, PyObject *type) {
  Vector v;
  if (t == Py_None) return v;
  v.given = true;
  v.n = call_int(t, m_numel);
  if (!is_contiguous(t)) {
    PyErr_Format(PyExc_ValueError, "%s is not contiguous", name);
    throw Failed{};
  }
  check_type(name, t, type);
  v.p = reinterpret_cast<void *>(call_int(t, m_data_ptr));
  return v;
}

void need(const char *name, const Vector &v, int64_t n) {
  if (!v.given || v.n >= n) return;
  PyErr_Format(PyExc_ValueError, "%s has %lld elements for %lld", name, (long long)v.n, (long long)n);
  throw Failed{};
}

// group_offsets and the number of groups that it bounds
const int32_t *offsets(PyObject *t, int &E, int without) {
  E = without;
  if (t == Py_None) return nullptr;
  const Vector v = vector("group_offsets", t, t_i32);
  E = as_int32(v.n - 1);
  return v.as<const int32_t>();
}

int64_t blocks32(int64_t cols) { return (cols + 31) / 32; }

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
    const Matrix x = matrix("x", a[0], t_bf16, true), q = matrix("q", a[1], t_u8),
                 s = matrix("scales", a[2], t_bf16);
    const int cols = as_int32(x.cols);
    need("q", q, x.rows, cols);
    need("scales", s, x.rows, blocks32(cols));
    int E;
    const int32_t *off = offsets(a[3], E, 0);
    const moe_stream_t st = stream(a[4]);
    return unlocked([=] {
      return moe_act8_quantize(x.as<uint16_t>(), x.ld, x.rows, cols, off, E, q.as<int8_t>(), q.ld,
                               s.as<uint16_t>(), s.ld, st);
    });
  });
}

// q, scales, x, group_offsets, stream
PyObject *act8_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<5>(args, n, [](PyObject *const *a) {
    const Matrix q = matrix("q", a[0], t_u8), s = matrix("scales", a[1], t_bf16),
                 x = matrix("x", a[2], t_bf16, true);
    const int cols = as_int32(x.cols);
    need("q", q, x.rows, cols);
    need("scales", s, x.rows, blocks32(cols));
    int E;
    const int32_t *off = offsets(a[3], E, 0);
    const moe_stream_t st = stream(a[4]);
    return unlocked([=] {
      return moe_act8_dequantize(q.as<int8_t>(), q.ld, s.as<uint16_t>(), s.ld, x.rows, cols, off, E,
                                 x.as<uint16_t>(), x.ld, st);
    });
  });
}

// h, act, q, scales, group_offsets, stream
PyObject *act8_swiglu_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject *const *a) {
    const Matrix h = matrix("h", a[0], t_bf16), act = matrix("act", a[1], t_bf16, true),
                 q = matrix("q", a[2], t_u8), s = matrix("scales", a[3], t_bf16);
    const int64_t rows = act.rows;
    const int F = as_int32(act.cols);
    need("h", h, rows, 2 * act.cols);
    need("q", q, rows, 2 * act.cols);
    need("scales", s, rows, 2 * blocks32(F));
    int E;
    const int32_t *off = offsets(a[4], E, 0);
    const moe_stream_t st = stream(a[5]);
    return unlocked([=] {
      return moe_act8_swiglu_fwd(h.as<uint16_t>(), h.ld, rows, F, off, E, act.as<uint16_t>(), act.ld,
                                 q.as<int8_t>(), q.ld, s.as<uint16_t>(), s.ld, st);
    });
  });
}

// q, scales, dact, dh, act, group_offsets, stream
PyObject *act8_swiglu_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<7>(args, n, [](PyObject *const *a) {
    const Matrix q = matrix("q", a[0], t_u8), s = matrix("scales", a[1], t_bf16),
                 dact = matrix("dact", a[2], t_bf16, true), dh = matrix("dh", a[3], t_bf16);
    const int64_t rows = dact.rows;
    const int F = as_int32(dact.cols);
    need("q", q, rows, 2 * dact.cols);
    need("scales", s, rows, 2 * blocks32(F));
    need("dh", dh, rows, 2 * dact.cols);
    Matrix act = {nullptr, 0, 0, 0};
    if (a[4] != Py_None) {
      act = matrix("act", a[4], t_bf16);
      need("act", act, rows, F);
    }
    int E;
    const int32_t *off = offsets(a[5], E, 0);
    const moe_stream_t st = stream(a[6]);
    return unlocked([=] {
      return moe_act8_swiglu_bwd(q.as<int8_t>(), q.ld, s.as<uint16_t>(), s.ld, dact.as<uint16_t>(),
                                 dact.ld, rows, F, off, E, dh.as<uint16_t>(), dh.ld,
                                 act.as<uint16_t>(), act.ld, st);
    });
  });
}

// An NVFP4 quantiser's fp32 scales: one, or one an expert of weights (MXFP4 reads none).
Vector fp4_scale(PyObject *t, int fmt, int map, int E) {
  const Vector v = vector("scale", t, t_f32);
  if (fmt == MOE_FP4_NV) need("scale", v, map == MOE_FP4_ROWS_GROUPED ? 1 : E);
  return v;
}

// x, fmt, q, sf, row_map, group_offsets, groups, row_index, index_div, scale, workspace,
// dev_status, stream
PyObject *fp4_quantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<13>(args, n, [](PyObject *const *a) {
    const int fmt = int32_arg(a[1]), map = int32_arg(a[4]), div = int32_arg(a[8]);
    const Matrix x = matrix("x", a[0], t_bf16, true), q = matrix("q", a[2], t_u8);
    const int cols = as_int32(x.cols);
    const int64_t rows = q.rows;
    need("q", q, rows, cols / 2);
    int E;
    const int32_t *off = offsets(a[5], E, int32_arg(a[6]));
    const Vector sf = vector("sf", a[3], t_u8), index = vector("row_index", a[7], t_i32),
                 scale = fp4_scale(a[9], fmt, map, E), ws = vector("workspace", a[10], t_u8),
                 status = vector("dev_status", a[11], t_i32);
    need("row_index", index, rows);
    need("dev_status", status, 1);
    const moe_stream_t st = stream(a[12]);
    return unlocked([=] {
      return moe_fp4_quantize(x.as<uint16_t>(), x.ld, x.rows, index.as<int32_t>(), div, rows, cols,
                              fmt, map, off, E, scale.as<float>(), q.as<uint8_t>(), q.ld,
                              sf.as<uint8_t>(), (size_t)sf.n, ws.p, (size_t)ws.n,
                              status.as<int32_t>(), st);
    });
  });
}

// q, sf, fmt, x, row_map, group_offsets, groups, scale, stream
PyObject *fp4_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<9>(args, n, [](PyObject *const *a) {
    const int fmt = int32_arg(a[2]), map = int32_arg(a[4]);
    const Matrix q = matrix("q", a[0], t_u8), x = matrix("x", a[3], t_bf16, true);
    const int cols = as_int32(x.cols);
    need("q", q, x.rows, cols / 2);
    int E;
    const int32_t *off = offsets(a[5], E, int32_arg(a[6]));
    const Vector sf = vector("sf", a[1], t_u8), scale = fp4_scale(a[7], fmt, map, E);
    const moe_stream_t st = stream(a[8]);
    return unlocked([=] {
      return moe_fp4_dequantize(q.as<uint8_t>(), q.ld, sf.as<uint8_t>(), (size_t)sf.n, x.rows, cols,
                                fmt, map, off, E, scale.as<float>(), x.as<uint16_t>(), x.ld, st);
    });
  });
}

// addresses of moe_fp4_weights and moe_fp4_buffers, x, sorted_to_flat, k, group_offsets, stream
PyObject *fp4_experts(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<7>(args, n, [](PyObject *const *a) {
    const auto w = reinterpret_cast<const moe_fp4_weights *>(as_int(a[0]));
    const auto b = reinterpret_cast<const moe_fp4_buffers *>(as_int(a[1]));
    const Matrix x = matrix("x", a[2], t_bf16, true);
    const int tokens = as_int32(x.rows), k = int32_arg(a[4]);
    const Vector s2f = vector("sorted_to_flat", a[3], t_i32),
                 off = vector("group_offsets", a[5], t_i32);
    if (w != nullptr && b != nullptr) {
      need("x", x, tokens, w->d);
      need("sorted_to_flat", s2f, b->rows_cap);
      need("group_offsets", off, (int64_t)w->E + 1);
    }
    const moe_stream_t st = stream(a[6]);
    return unlocked([=] {
      return moe_fp4_experts(w, b, x.as<uint16_t>(), x.ld, tokens, s2f.as<int32_t>(), k,
                             off.as<int32_t>(), st);
    });
  });
}

// A, sfa, B, sfb, fmt, group_offsets, K (under 0: of B), epilogue, C, Q2, sf2, a_scale, b_scale,
// q2_scale, dev_status, stream
PyObject *gmm_fp4(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<16>(args, n, [](PyObject *const *a) {
    const int fmt = int32_arg(a[4]), epilogue = int32_arg(a[7]);
    const bool swiglu = epilogue == MOE_EPI_SWIGLU_FWD;
    const Matrix A = matrix("A", a[0], t_u8), B = matrix("B", a[2], t_u8);
    int E;
    int64_t stride_b;
    {
      Tuple shape(m_shape.get(a[2])), stride(m_stride.call(a[2]));
      if (PyTuple_GET_SIZE(shape.o) != 3) {
        PyErr_SetString(PyExc_ValueError, "B is [E, N, K / 2]");
        throw Failed{};
      }
      E = as_int32(item(shape.o, 0));
      stride_b = item(stride.o, 0);
    }
    int K = int32_arg(a[6]);
    if (K < 0) K = as_int32(2 * B.cols);
    const int N = as_int32(B.rows);
    const int64_t rows = A.rows;
    need("A", A, rows, K / 2);
    need("B", B, N, K / 2);
    Matrix C = {nullptr, 0, 0, 0}, Q2 = C;
    int c_dtype = MOE_DTYPE_BF16;
    if (a[8] != Py_None) {
      PyObject *d = m_dtype.get(a[8]);
      if (d == nullptr) throw Failed{};
      Py_DECREF(d);  // (the type lives on)
      if (d == t_f32) c_dtype = MOE_DTYPE_F32;
      C = matrix("C", a[8], d == t_f32 ? t_f32 : t_bf16);
      need("C", C, rows, N);
    }
    if (a[9] != Py_None) {
      Q2 = matrix("Q2", a[9], t_u8);
      if (swiglu) need("Q2", Q2, rows, N / 4);
    }
    const Vector sfa = vector("sfa", a[1], t_u8), sfb = vector("sfb", a[3], t_u8),
                 off = vector("group_offsets", a[5], t_i32), sf2 = vector("sf2", a[10], t_u8),
                 ga = vector("a_scale", a[11], t_f32), gb = vector("b_scale", a[12], t_f32),
                 g2 = vector("q2_scale", a[13], t_f32), status = vector("dev_status", a[14], t_i32);
    need("sfa", sfa, moe_fp4_scale_bytes(rows, K, fmt, MOE_FP4_ROWS_GROUPED, E));
    need("sfb", sfb, moe_fp4_scale_bytes((int64_t)E * N, K, fmt,
                                         swiglu ? MOE_FP4_ROWS_SWIGLU : MOE_FP4_ROWS_EXPERTS, E));
    need("group_offsets", off, (int64_t)E + 1);
    need("a_scale", ga, 1);
    need("b_scale", gb, E);
    need("q2_scale", g2, 1);
    need("dev_status", status, 1);
    const moe_stream_t st = stream(a[15]);
    return unlocked([=] {
      return moe_gmm_fp4(A.as<uint8_t>(), A.ld, sfa.as<uint8_t>(), ga.as<float>(), B.as<uint8_t>(),
                         B.ld, stride_b, sfb.as<uint8_t>(), gb.as<float>(), fmt, off.as<int32_t>(), E,
                         rows, K, N, epilogue, C.p, c_dtype, C.ld, Q2.as<uint8_t>(), Q2.ld,
                         sf2.as<uint8_t>(), (size_t)sf2.n, g2.as<float>(), status.as<int32_t>(), st);
    });
  });
}

// ------------------------------------------------ around the expert layer
float float_arg(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed{};
  return (float)v;
}

// `name` of the call, if given, lies on GPU `dev`.
void on_device(const char *name, PyObject *t, int64_t dev) {
  if (t == Py_None) return;
  PyObject *r = m_get_device.call(t);
  if (r == nullptr) throw Failed{};
  const long long at = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (at == dev && at >= 0) return;
  if (!PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, at < 0 ? "%s is not on a GPU" : "%s is on GPU %lld, the call on %lld",
                 name, at, (long long)dev);
  throw Failed{};
}

// MOE_DTYPE_* of a tensor that may be bf16 or fp32.
int real_type(const char *name, PyObject *t) {
  PyObject *d = m_dtype.get(t);
  if (d == nullptr) throw Failed{};
  const bool f32 = d == t_f32, ok = f32 || d == t_bf16;
  if (!ok) PyErr_Format(PyExc_ValueError, "%s is %S, not %S or %S", name, d, t_bf16, t_f32);
  Py_DECREF(d);
  if (!ok) throw Failed{};
  return f32 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16;
}

PyObject *type_object(int dtype) { return dtype == MOE_DTYPE_F32 ? t_f32 : t_bf16; }

// A matrix that may be None; given, of [rows, cols] (rows < 0: any, which it then sets).
Matrix optional(const char *name, PyObject *t, PyObject *type, int64_t &rows, int64_t &cols) {
  if (t == Py_None) return {nullptr, 0, 0, 0};
  const Matrix m = matrix(name, t, type, true);
  if (rows < 0) {
    rows = m.rows;
    cols = m.cols;
  } else if (m.rows != rows || m.cols != cols) {
    PyErr_Format(PyExc_ValueError, "%s is [%lld, %lld], not [%lld, %lld]", name, (long long)m.rows,
                 (long long)m.cols, (long long)rows, (long long)cols);
    throw Failed{};
  }
  return m;
}

// x, residual, w, eps, h, y, codes, q, scales, device, stream
PyObject *rms_norm(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<11>(args, n, [](PyObject *const *a) {
    int64_t rows = -1, cols = 0;
    const Matrix x = optional("x", a[0], t_bf16, rows, cols);
    const int dtype = a[1] != Py_None   ? real_type("residual", a[1])
                      : a[4] != Py_None ? real_type("h", a[4])
                                        : MOE_DTYPE_BF16;
    const Matrix res = optional("residual", a[1], type_object(dtype), rows, cols),
                 h = optional("h", a[4], type_object(dtype), rows, cols),
                 y = optional("y", a[5], t_bf16, rows, cols);
    if (a[0] == Py_None && a[1] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "neither x nor residual");
      throw Failed{};
    }
    const int wt = real_type("w", a[2]);
    const Vector w = vector("w", a[2], type_object(wt));
    need("w", w, cols);
    const float eps = float_arg(a[3]);
    const int codes = int32_arg(a[6]), c = as_int32(cols);
    Matrix q = {nullptr, 0, 0, 0}, s = q;
    size_t bytes = 0;
    if (codes != MOE_CODES_NONE) {
      q = optional("q", a[7], t_u8, rows, cols);
      if (a[8] != Py_None && codes == MOE_CODES_ACT8) {
        s = matrix("scales", a[8], t_bf16, true);
        need("scales", s, rows, blocks32(cols));
        bytes = s.rows > 0 ? 2 * (size_t)((s.rows - 1) * s.ld + s.cols) : 0;
      } else {
        const Vector v = vector("scales", a[8], t_u8);
        s.p = v.p;
        bytes = (size_t)v.n;
      }
    }
    const int64_t dev = as_int(a[9]);
    const char *names[] = {"x", "residual", "w", nullptr, "h", "y", nullptr, "q", "scales"};
    for (int i = 0; i < 9; ++i)
      if (names[i] != nullptr && (i < 7 || codes != MOE_CODES_NONE)) on_device(names[i], a[i], dev);
    const moe_stream_t st = stream(a[10]);
    return unlocked([=] {
      return moe_rms_norm(x.as<uint16_t>(), x.ld, res.p, res.ld, dtype, rows, c, w.p, wt, eps, h.p,
                          h.ld, y.as<uint16_t>(), y.ld, codes, q.as<uint8_t>(), q.ld, s.p, s.ld, bytes,
                          st);
    });
  });
}

// dy, h, w, eps, d_residual, dh, dx, dw, accumulate, workspace, device, stream
PyObject *rms_norm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<12>(args, n, [](PyObject *const *a) {
    int64_t rows = -1, cols = 0;
    const Matrix dy = optional("dy", a[0], t_bf16, rows, cols);
    if (a[0] == Py_None || a[5] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "dy and dh are needed");
      throw Failed{};
    }
    const int dtype = real_type("h", a[1]);
    const Matrix h = optional("h", a[1], type_object(dtype), rows, cols),
                 res = optional("d_residual", a[4], type_object(dtype), rows, cols),
                 dh = optional("dh", a[5], type_object(dtype), rows, cols),
                 dx = optional("dx", a[6], t_bf16, rows, cols);
    const int wt = real_type("w", a[2]);
    const Vector w = vector("w", a[2], type_object(wt)), dw = vector("dw", a[7], t_f32),
                 ws = vector("workspace", a[9], t_u8);
    need("w", w, cols);
    need("dw", dw, cols);
    const float eps = float_arg(a[3]);
    const int c = as_int32(cols), accumulate = int32_arg(a[8]);
    const int64_t dev = as_int(a[10]);
    const char *names[] = {"dy", "h", "w", nullptr, "d_residual", "dh", "dx", "dw", nullptr, "workspace"};
    for (int i = 0; i < 10; ++i)
      if (names[i] != nullptr) on_device(names[i], a[i], dev);
    const moe_stream_t st = stream(a[11]);
    return unlocked([=] {
      return moe_rms_norm_bwd(dy.as<uint16_t>(), dy.ld, h.p, h.ld, dtype, rows, c, w.p, wt, eps, res.p,
                              res.ld, dh.p, dh.ld, dx.as<uint16_t>(), dx.ld, dw.as<float>(), accumulate,
                              ws.p, (size_t)ws.n, st);
    });
  });
}

// q, sf, fmt, x, device, stream
PyObject *mx_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<6>(args, n, [](PyObject *const *a) {
    const Matrix q = matrix("q", a[0], t_u8, true), x = matrix("x", a[3], t_bf16, true);
    need("q", q, x.rows, x.cols);
    const Vector sf = vector("sf", a[1], t_u8);
    const int fmt = int32_arg(a[2]), cols = as_int32(x.cols);
    const int64_t dev = as_int(a[4]);
    on_device("q", a[0], dev);
    on_device("sf", a[1], dev);
    on_device("x", a[3], dev);
    const moe_stream_t st = stream(a[5]);
    return unlocked([=] {
      return moe_mx_dequantize(q.as<uint8_t>(), q.ld, sf.as<uint8_t>(), (size_t)sf.n, x.rows, cols, fmt,
                               x.as<uint16_t>(), x.ld, st);
    });
  });
}

// What the two calls of the sequences' loss have in common.
struct SeqAux {
  Matrix logits, d_logits = {nullptr, 0, 0, 0};
  Vector offsets, mask, counts, tokens;
  int T, E, B, score_fn, accumulate;
  float coeff, z_coeff, d_loss;
  SeqAux(PyObject *l, PyObject *off, PyObject *m, PyObject *fn, PyObject *c, PyObject *z, PyObject *cnt,
         PyObject *tok, PyObject *dl, PyObject *d, PyObject *acc)
      : logits(matrix("logits", l, t_f32, true)), offsets(vector("seq_offsets", off, t_i32)),
        mask(vector("token_mask", m, t_u8)), counts(vector("counts", cnt, t_i32)),
        tokens(vector("tokens", tok, t_i32)), T(as_int32(logits.rows)), E(as_int32(logits.cols)),
        B(as_int32(offsets.n - 1)), score_fn(int32_arg(fn)), accumulate(int32_arg(acc)),
        coeff(float_arg(c)), z_coeff(float_arg(z)), d_loss(float_arg(dl)) {
    int64_t rows = T, cols = E;
    d_logits = optional("d_logits", d, t_f32, rows, cols);
    need("token_mask", mask, T);
    need("counts", counts, (int64_t)B * E);
    need("tokens", tokens, B);
  }
  static void on(int64_t dev, PyObject *l, PyObject *off, PyObject *m, PyObject *cnt, PyObject *tok,
                 PyObject *d) {
    on_device("logits", l, dev);
    on_device("seq_offsets", off, dev);
    on_device("token_mask", m, dev);
    on_device("counts", cnt, dev);
    on_device("tokens", tok, dev);
    on_device("d_logits", d, dev);
  }
};

// logits, topk_idx, seq_offsets, token_mask, score_fn, coeff, z_coeff, counts, tokens, probs_mean,
// loss, d_loss, d_logits, accumulate, workspace, device, stream
PyObject *seq_aux_loss(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<17>(args, n, [](PyObject *const *a) {
    const int64_t dev = as_int(a[15]);
    const Matrix idx = matrix("topk_idx", a[1], t_i32, true);
    const Vector flat = vector("topk_idx", a[1], t_i32), probs = vector("probs_mean", a[9], t_f32),
                 loss = vector("loss", a[10], t_f32), ws = vector("workspace", a[14], t_u8);
    const SeqAux s(a[0], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[11], a[12], a[13]);
    const int k = as_int32(idx.cols);
    if (idx.rows != s.T) {
      PyErr_Format(PyExc_ValueError, "topk_idx of %lld tokens, logits of %d", (long long)idx.rows, s.T);
      throw Failed{};
    }
    need("probs_mean", probs, (int64_t)s.B * s.E);
    need("loss", loss, 2);
    SeqAux::on(dev, a[0], a[2], a[3], a[7], a[8], a[12]);
    on_device("topk_idx", a[1], dev);
    on_device("probs_mean", a[9], dev);
    on_device("loss", a[10], dev);
    on_device("workspace", a[14], dev);
    const moe_stream_t st = stream(a[16]);
    return unlocked([&] {
      return moe_seq_aux_loss(s.logits.as<float>(), s.logits.ld, s.T, s.E, k, s.score_fn,
                              flat.as<int32_t>(), s.offsets.as<int32_t>(), s.B, s.mask.as<uint8_t>(),
                              s.coeff, s.z_coeff, s.counts.as<int32_t>(), s.tokens.as<int32_t>(),
                              probs.as<float>(), loss.as<float>(), s.d_loss, s.d_logits.as<float>(),
                              s.d_logits.ld, s.accumulate, ws.p, (size_t)ws.n, st);
    });
  });
}

// logits, k, seq_offsets, token_mask, score_fn, coeff, z_coeff, counts, tokens, d_loss, d_logits,
// accumulate, device, stream
PyObject *seq_aux_loss_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<14>(args, n, [](PyObject *const *a) {
    const SeqAux s(a[0], a[2], a[3], a[4], a[5], a[6], a[7], a[8], a[9], a[10], a[11]);
    const int k = int32_arg(a[1]);
    SeqAux::on(as_int(a[12]), a[0], a[2], a[3], a[7], a[8], a[10]);
    const moe_stream_t st = stream(a[13]);
    return unlocked([&] {
      return moe_seq_aux_loss_bwd(s.logits.as<float>(), s.logits.ld, s.T, s.E, k, s.score_fn,
                                  s.offsets.as<int32_t>(), s.B, s.mask.as<uint8_t>(), s.coeff,
                                  s.z_coeff, s.counts.as<int32_t>(), s.tokens.as<int32_t>(), s.d_loss,
                                  s.d_logits.as<float>(), s.d_logits.ld, s.accumulate, st);
    });
  });
}

// plan, chunks, max_norm (None: the norm alone), scale, norm, workspace, device, stream
PyObject *clip_grads(PyObject *, PyObject *const *args, Py_ssize_t n) {
  return entry<8>(args, n, [](PyObject *const *a) {
    const Vector plan = vector("plan", a[0], t_u8), norm = vector("norm", a[4], t_f32),
                 ws = vector("workspace", a[5], t_u8);
    const int64_t chunks = as_int(a[1]), dev = as_int(a[6]);
    if (chunks < 0 || plan.n / 32 < chunks) {
      PyErr_Format(PyExc_ValueError, "a plan of %lld bytes for %lld chunks", (long long)plan.n,
                   (long long)chunks);
      throw Failed{};
    }
    need("norm", norm, 1);
    const float scale = float_arg(a[3]), most = a[2] == Py_None ? 0.0f : float_arg(a[2]);
    const bool clip = a[2] != Py_None;
    on_device("plan", a[0], dev);
    on_device("norm", a[4], dev);
    on_device("workspace", a[5], dev);
    const moe_stream_t st = stream(a[7]);
    return unlocked([=] {
      return clip ? moe_clip_grads(plan.p, chunks, most, scale, norm.as<float>(), ws.p, (size_t)ws.n, st)
                  : moe_grad_norm(plan.p, chunks, scale, norm.as<float>(), ws.p, (size_t)ws.n, st);
    });
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
    {"gmm_fp4", fast(gmm_fp4), METH_FASTCALL, nullptr},
    {"fp4_experts", fast(fp4_experts), METH_FASTCALL, nullptr},
    {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
    {"rms_norm_bwd", fast(rms_norm_bwd), METH_FASTCALL, nullptr},
    {"mx_dequantize", fast(mx_dequantize), METH_FASTCALL, nullptr},
    {"seq_aux_loss", fast(seq_aux_loss), METH_FASTCALL, nullptr},
    {"seq_aux_loss_bwd", fast(seq_aux_loss_bwd), METH_FASTCALL, nullptr},
    {"clip_grads", fast(clip_grads), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) {
  PyObject *torch = PyImport_ImportModule("torch");
  if (torch == nullptr) return nullptr;
  PyObject *tensor = PyObject_GetAttrString(torch, "Tensor");
  struct {
    PyObject **o;
    const char *name;
  } const types[] = {{&t_bf16, "bfloat16"}, {&t_u8, "uint8"}, {&t_i8, "int8"}, {&t_i32, "int32"},
                     {&t_f32, "float32"}};
  bool ok = tensor != nullptr && PyType_Check(tensor);
  for (const auto &n : types) ok = ok && (*n.o = PyObject_GetAttrString(torch, n.name)) != nullptr;
  Py_DECREF(torch);
  if (!ok) return nullptr;
  tensor_type = (PyTypeObject *)tensor;
  for (Member *m : {&m_data_ptr, &m_stride, &m_numel, &m_shape, &m_is_contiguous, &m_dtype, &m_get_device}) {
    m->name = PyUnicode_InternFromString(m->text);
    m->descr = PyObject_GetAttrString(tensor, m->text);
    if (m->name == nullptr || m->descr == nullptr) return nullptr;
  }
  return PyModule_Create(&module);
}
