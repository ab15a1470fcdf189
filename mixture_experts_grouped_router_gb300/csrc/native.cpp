// Python calls of the short low-bit operators: the tensors' pointers, sizes and
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
       m_is_contiguous = {"is_contiguous"}, m_dtype = {"dtype"};

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
  for (Member *m : {&m_data_ptr, &m_stride, &m_numel, &m_shape, &m_is_contiguous, &m_dtype}) {
    m->name = PyUnicode_InternFromString(m->text);
    m->descr = PyObject_GetAttrString(tensor, m->text);
    if (m->name == nullptr || m->descr == nullptr) return nullptr;
  }
  return PyModule_Create(&module);
}
