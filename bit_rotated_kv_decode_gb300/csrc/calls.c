/* Argument marshalling of the paged-cache calls for Python, in C.
 *
 * These calls are made for every layer of a decode step, and reading eight tensors'
 * attributes and converting twenty arguments took Python 7.6 of a call's 11 us.  Each
 * function here checks its tensors (type, device, layout, shape) and makes the C call;
 * it returns the call's status, or None where anything is not as the fast case has it
 * (a wrong tensor, no workspace, a sequence that is no list or tuple).  The caller then
 * takes the same steps in Python, which says what is wrong.  Nothing is kept between
 * calls but what setup() gave. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "oscar.h"

#define MAX_REQ 256
#define HEAD_DIM 128

typedef oscar_status (*append16_fn)(void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t,
                                    int32_t, int32_t, const oscar_rope*, const uint16_t*, int64_t, const uint16_t*,
                                    int64_t, const uint16_t*, int64_t, uint16_t*, int32_t*, void*);
typedef oscar_status (*append4_fn)(void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t,
                                   int32_t, int32_t, int32_t, const oscar_rope*, const uint16_t*, int64_t,
                                   const uint16_t*, int64_t, const uint16_t*, int64_t, uint16_t*, int32_t*, void*);
typedef oscar_status (*read4_fn)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                 int32_t, int32_t, int32_t, void*, void*, int32_t, int32_t*, void*);
typedef oscar_status (*attend16_fn)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                    int32_t, int32_t, int32_t, int32_t, int32_t, float, const uint16_t*, int64_t, void*,
                                    int32_t, float*, int32_t*, void*, size_t, void*);
typedef oscar_status (*attend4_fn)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                   int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, float, const uint16_t*,
                                   int64_t, void*, int32_t, float*, int32_t*, void*, size_t, void*);

static struct {
  PyObject *bf16, *f32, *i32, *u8;         /* torch's type objects */
  PyObject *get_device, *raw_stream;       /* current device, current stream of a device */
  PyObject *n_dtype, *n_device, *n_contiguous, *n_shape, *n_ptr, *n_stride;   /* attribute names */
  append16_fn append16;
  append4_fn append4;
  read4_fn read4;
  attend16_fn attend16;
  attend4_fn attend4;
} g;

/* -1 in a shape: any extent, written back */
typedef struct {
  void* ptr;
  int64_t shape[5];
} Tensor;

static int as_long(PyObject* o, long long* out) {   /* steals o */
  if (!o) {
    PyErr_Clear();
    return 0;
  }
  *out = PyLong_AsLongLong(o);
  Py_DECREF(o);
  if (*out == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return 1;
}

static int same_attr(PyObject* t, PyObject* name, PyObject* want) {
  PyObject* a = PyObject_GetAttr(t, name);
  if (!a) {
    PyErr_Clear();
    return 0;
  }
  const int same = a == want;
  Py_DECREF(a);
  return same;
}

static int shape_of(PyObject* t, int dims, Tensor* out) {
  PyObject* s = PyObject_GetAttr(t, g.n_shape);
  if (!s) {
    PyErr_Clear();
    return 0;
  }
  int ok = PyTuple_Check(s) && PyTuple_GET_SIZE(s) == dims;
  for (int i = 0; ok && i < dims; ++i) {
    const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(s, i));
    ok = v >= 0 && (out->shape[i] < 0 || out->shape[i] == v);
    out->shape[i] = v;
  }
  Py_DECREF(s);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return ok;
}

/* type, device and shape (dims 0: any) of a tensor, and its address */
static int tensor(PyObject* t, PyObject* dtype, long long device, int dims, Tensor* out) {
  long long d, p;
  if (!same_attr(t, g.n_dtype, dtype) || !as_long(PyObject_CallMethodNoArgs(t, g.n_device), &d) || d != device) return 0;
  if (dims && !shape_of(t, dims, out)) return 0;
  if (!as_long(PyObject_CallMethodNoArgs(t, g.n_ptr), &p)) return 0;
  out->ptr = (void*)(uintptr_t)p;
  return 1;
}

static int dense(PyObject* t, PyObject* dtype, long long device, int dims, Tensor* out) {
  PyObject* c = PyObject_CallMethodNoArgs(t, g.n_contiguous);
  if (!c) {
    PyErr_Clear();
    return 0;
  }
  const int yes = c == Py_True;
  Py_DECREF(c);
  return yes && tensor(t, dtype, device, dims, out);
}

/* bf16 [rows][heads][128] whose heads lie densely; heads < 0: any */
static int heads_of(PyObject* t, long long device, int64_t rows, int64_t heads, Tensor* out, int64_t* stride) {
  out->shape[0] = rows;
  out->shape[1] = heads;
  out->shape[2] = HEAD_DIM;
  if (!tensor(t, g.bf16, device, 3, out)) return 0;
  PyObject* s = PyObject_CallMethodNoArgs(t, g.n_stride);
  if (!s) {
    PyErr_Clear();
    return 0;
  }
  int ok = 0;
  if (PyTuple_Check(s) && PyTuple_GET_SIZE(s) == 3) {
    const long long a = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 0)), b = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 1)),
                    c = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 2));
    ok = !PyErr_Occurred() && c == 1 && (b == HEAD_DIM || out->shape[1] <= 1);
    *stride = rows > 1 ? a : out->shape[1] * HEAD_DIM;
  }
  PyErr_Clear();
  Py_DECREF(s);
  return ok;
}

/* host ints of a list or tuple of n, not negative; their sum, or -1 */
static int64_t counts(PyObject* o, Py_ssize_t n, int32_t* out) {
  if (!(PyList_Check(o) || PyTuple_Check(o)) || PySequence_Fast_GET_SIZE(o) != n) return -1;
  int64_t sum = 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* v = PySequence_Fast_GET_ITEM(o, i);
    if (!PyLong_CheckExact(v)) return -1;
    const long long x = PyLong_AsLongLong(v);
    if (x < 0 || x > INT32_MAX) {
      PyErr_Clear();
      return -1;
    }
    out[i] = (int32_t)x;
    sum += x;
  }
  return sum;
}

static int context(PyObject* stream, long long* device, void** raw) {
  long long s;
  if (stream != Py_None || !g.get_device) return 0;
  if (!as_long(PyObject_CallNoArgs(g.get_device), device)) return 0;
  PyObject* d = PyLong_FromLongLong(*device);
  if (!d) {
    PyErr_Clear();
    return 0;
  }
  const int ok = as_long(PyObject_CallOneArg(g.raw_stream, d), &s);
  Py_DECREF(d);
  *raw = (void*)(uintptr_t)s;
  return ok;
}

static long group_of(PyObject* o) {   /* -1: no int */
  const long v = PyLong_AsLong(o);
  if (v == -1) PyErr_Clear();
  return v;
}

static Py_ssize_t requests(PyObject* lens) {
  if (!(PyList_Check(lens) || PyTuple_Check(lens))) return 0;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(lens);
  return n <= MAX_REQ ? n : 0;
}

static int pool_of(PyObject* kv, long group, long long device, int64_t hkv, Tensor* out) {
  out->shape[0] = -1;
  out->shape[1] = hkv;
  if (group == 0) {
    out->shape[2] = 2;
    out->shape[3] = 64;
    out->shape[4] = HEAD_DIM;
    return dense(kv, g.bf16, device, 5, out);
  }
  if (group != 128 && group != 64) return 0;
  out->shape[2] = group == 128 ? 8704 : 9216;
  return dense(kv, g.u8, device, 3, out);
}

/* append(group, kv, page_table, lens, k, v, rope, q, q_out, new_lens, interleaved, error, stream) */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  (void)self;
  int32_t lens[MAX_REQ], news[MAX_REQ];
  long long device;
  void* stream;
  if (count != 13 || !context(a[12], &device, &stream)) Py_RETURN_NONE;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || counts(a[3], n, lens) < 0) Py_RETURN_NONE;
  int64_t rows = n;
  if (a[9] != Py_None && (rows = counts(a[9], n, news)) < 0) Py_RETURN_NONE;
  Tensor kv, table = {0, {n, -1}}, k, v, q = {0}, qo = {0}, rope = {0, {-1, -1}}, err = {0};
  int64_t ks, vs, qs = 0;
  if (!heads_of(a[4], device, rows, -1, &k, &ks)) Py_RETURN_NONE;
  const int64_t hkv = k.shape[1];
  if (!heads_of(a[5], device, rows, hkv, &v, &vs) || !pool_of(a[1], group, device, hkv, &kv) ||
      !dense(a[2], g.i32, device, 2, &table))
    Py_RETURN_NONE;
  int64_t hq = 0;
  if (a[7] != Py_None && a[8] != Py_None) {
    if (!heads_of(a[7], device, rows, -1, &q, &qs)) Py_RETURN_NONE;
    hq = q.shape[1];
    qo.shape[0] = rows;
    qo.shape[1] = hq;
    qo.shape[2] = HEAD_DIM;
    if (!dense(a[8], g.bf16, device, 3, &qo)) Py_RETURN_NONE;
  } else if (a[7] != a[8]) {
    Py_RETURN_NONE;
  }
  oscar_rope r;
  const oscar_rope* rp = 0;
  if (a[6] != Py_None) {
    if (!dense(a[6], g.f32, device, 2, &rope) || rope.shape[0] > INT32_MAX || rope.shape[1] > INT32_MAX) Py_RETURN_NONE;
    const int inter = PyObject_IsTrue(a[10]);
    if (inter < 0) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    r.table = (const float*)rope.ptr;
    r.length = (int32_t)rope.shape[0];
    r.dim = (int32_t)rope.shape[1];
    r.interleaved = inter;
    rp = &r;
  }
  if (a[11] != Py_None && !dense(a[11], g.i32, device, 0, &err)) Py_RETURN_NONE;
  if (table.shape[1] > INT32_MAX || hkv > INT32_MAX || hq > INT32_MAX) Py_RETURN_NONE;
  if (rows == 0) return PyLong_FromLong(OSCAR_OK);
  const int32_t* nl = a[9] == Py_None ? 0 : news;
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  if (group == 0)
    st = g.append16(kv.ptr, kv.shape[0], (const int32_t*)table.ptr, (int32_t)table.shape[1], lens, nl, (int32_t)n,
                    (int32_t)hq, (int32_t)hkv, rp, (const uint16_t*)q.ptr, qs, (const uint16_t*)k.ptr, ks,
                    (const uint16_t*)v.ptr, vs, (uint16_t*)qo.ptr, (int32_t*)err.ptr, stream);
  else
    st = g.append4(kv.ptr, kv.shape[0], (const int32_t*)table.ptr, (int32_t)table.shape[1], lens, nl, (int32_t)n,
                   (int32_t)hq, (int32_t)hkv, (int32_t)group, rp, (const uint16_t*)q.ptr, qs, (const uint16_t*)k.ptr,
                   ks, (const uint16_t*)v.ptr, vs, (uint16_t*)qo.ptr, (int32_t*)err.ptr, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* read(group, kv, page_table, starts, counts, k_out, v_out, error, stream) */
static PyObject* py_read(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  (void)self;
  int32_t starts[MAX_REQ], cnt[MAX_REQ];
  long long device;
  void* stream;
  if (count != 9 || !context(a[8], &device, &stream)) Py_RETURN_NONE;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || group == 0 || counts(a[3], n, starts) < 0) Py_RETURN_NONE;
  const int64_t rows = counts(a[4], n, cnt);
  Tensor kv, table = {0, {n, -1}}, ko = {0, {rows, -1, HEAD_DIM}}, vo, err = {0};
  if (rows < 0) Py_RETURN_NONE;
  const int f32 = same_attr(a[5], g.n_dtype, g.f32);
  PyObject* kind = f32 ? g.f32 : g.bf16;
  if (!dense(a[5], kind, device, 3, &ko)) Py_RETURN_NONE;
  const int64_t hkv = ko.shape[1];
  vo = ko;
  if (!dense(a[6], kind, device, 3, &vo) || !pool_of(a[1], group, device, hkv, &kv) ||
      !dense(a[2], g.i32, device, 2, &table) || table.shape[1] > INT32_MAX || hkv > INT32_MAX)
    Py_RETURN_NONE;
  if (a[7] != Py_None && !dense(a[7], g.i32, device, 0, &err)) Py_RETURN_NONE;
  if (rows == 0) return PyLong_FromLong(OSCAR_OK);
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  st = g.read4(kv.ptr, kv.shape[0], (const int32_t*)table.ptr, (int32_t)table.shape[1], starts, cnt, (int32_t)n,
               (int32_t)hkv, (int32_t)group, ko.ptr, vo.ptr, f32 ? OSCAR_F32 : OSCAR_BF16, (int32_t*)err.ptr, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* attend(group, kv, page_table, lens, q, out, num_kv_heads, window, sinks, q_lens, scale, lse, workspace, error,
 *        stream) */
static PyObject* py_attend(PyObject* self, PyObject* const* a, Py_ssize_t count) {
  (void)self;
  int32_t lens[MAX_REQ], ql[MAX_REQ];
  long long device;
  void* stream;
  if (count != 15 || a[12] == Py_None || !context(a[14], &device, &stream)) Py_RETURN_NONE;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || counts(a[3], n, lens) < 0) Py_RETURN_NONE;
  int64_t rows = n;
  if (a[9] != Py_None && (rows = counts(a[9], n, ql)) < 0) Py_RETURN_NONE;
  const long long hkv = PyLong_AsLongLong(a[6]), window = PyLong_AsLongLong(a[7]), sinks = PyLong_AsLongLong(a[8]);
  const double scale = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (hkv < 1 || hkv > INT32_MAX || window < INT32_MIN || window > INT32_MAX || sinks < 0 || sinks > INT32_MAX)
    Py_RETURN_NONE;
  Tensor kv, table = {0, {n, -1}}, q, out, lse = {0}, ws = {0, {-1}}, err = {0};
  int64_t qs;
  if (!heads_of(a[4], device, rows, -1, &q, &qs)) Py_RETURN_NONE;
  const int64_t hq = q.shape[1];
  const int f32 = same_attr(a[5], g.n_dtype, g.f32);
  out.shape[0] = lse.shape[0] = rows;
  out.shape[1] = lse.shape[1] = hq;
  out.shape[2] = HEAD_DIM;
  if (!dense(a[5], f32 ? g.f32 : g.bf16, device, 3, &out) || !pool_of(a[1], group, device, hkv, &kv) ||
      !dense(a[2], g.i32, device, 2, &table) || !dense(a[12], g.u8, device, 1, &ws) || table.shape[1] > INT32_MAX ||
      hq > INT32_MAX)
    Py_RETURN_NONE;
  if (a[11] != Py_None && !dense(a[11], g.f32, device, 2, &lse)) Py_RETURN_NONE;
  if (a[13] != Py_None && !dense(a[13], g.i32, device, 0, &err)) Py_RETURN_NONE;
  if (rows == 0) return PyLong_FromLong(OSCAR_OK);
  const int32_t* qn = a[9] == Py_None ? 0 : ql;
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  if (group == 0)
    st = g.attend16(kv.ptr, kv.shape[0], (const int32_t*)table.ptr, (int32_t)table.shape[1], lens, qn, (int32_t)n,
                    (int32_t)hq, (int32_t)hkv, (int32_t)window, (int32_t)sinks, (float)scale, (const uint16_t*)q.ptr, qs,
                    out.ptr, f32 ? OSCAR_F32 : OSCAR_BF16, (float*)lse.ptr, (int32_t*)err.ptr, ws.ptr,
                    (size_t)ws.shape[0], stream);
  else
    st = g.attend4(kv.ptr, kv.shape[0], (const int32_t*)table.ptr, (int32_t)table.shape[1], lens, qn, (int32_t)n,
                   (int32_t)hq, (int32_t)hkv, (int32_t)group, (int32_t)window, (int32_t)sinks, (float)scale,
                   (const uint16_t*)q.ptr, qs, out.ptr, f32 ? OSCAR_F32 : OSCAR_BF16, (float*)lse.ptr,
                   (int32_t*)err.ptr, ws.ptr, (size_t)ws.shape[0], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

/* setup((bf16, f32, i32, u8), (current device, raw stream), (five function addresses)) */
static PyObject* py_setup(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *types[4], *fns[2];
  unsigned long long at[5];
  if (!PyArg_ParseTuple(args, "(OOOO)(OO)(KKKKK)", &types[0], &types[1], &types[2], &types[3], &fns[0], &fns[1], &at[0],
                        &at[1], &at[2], &at[3], &at[4]))
    return 0;
  for (int i = 0; i < 4; ++i) Py_INCREF(types[i]);
  for (int i = 0; i < 2; ++i) Py_INCREF(fns[i]);
  g.bf16 = types[0], g.f32 = types[1], g.i32 = types[2], g.u8 = types[3];
  g.get_device = fns[0], g.raw_stream = fns[1];
  g.append16 = (append16_fn)(uintptr_t)at[0];
  g.append4 = (append4_fn)(uintptr_t)at[1];
  g.read4 = (read4_fn)(uintptr_t)at[2];
  g.attend16 = (attend16_fn)(uintptr_t)at[3];
  g.attend4 = (attend4_fn)(uintptr_t)at[4];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", py_setup, METH_VARARGS, 0},
                                {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, 0},
                                {"read", (PyCFunction)(void (*)(void))py_read, METH_FASTCALL, 0},
                                {"attend", (PyCFunction)(void (*)(void))py_attend, METH_FASTCALL, 0},
                                {0, 0, 0, 0}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_oscar_calls", 0, -1, methods, 0, 0, 0, 0};

PyMODINIT_FUNC PyInit__oscar_calls(void) {
  g.n_dtype = PyUnicode_InternFromString("dtype");
  g.n_device = PyUnicode_InternFromString("get_device");
  g.n_contiguous = PyUnicode_InternFromString("is_contiguous");
  g.n_shape = PyUnicode_InternFromString("shape");
  g.n_ptr = PyUnicode_InternFromString("data_ptr");
  g.n_stride = PyUnicode_InternFromString("stride");
  if (!g.n_dtype || !g.n_device || !g.n_contiguous || !g.n_shape || !g.n_ptr || !g.n_stride) return 0;
  return PyModule_Create(&module);
}
