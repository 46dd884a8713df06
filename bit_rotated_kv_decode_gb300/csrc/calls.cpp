// Argument marshalling of the paged-cache calls for Python, in C++.
//
// These calls are made for every layer of a decode step.  Reading eight tensors'
// attributes and converting twenty arguments took Python 7.6 of a call's 11 us; through
// the attributes' C calls it took 2.6 of 6.0, and with the tensors read directly it takes
// 0.4 of 3.6 (the launch is the rest).  Each function here checks
// its tensors (type, device, layout, shape) and makes the C call; it returns the call's
// status, or None where anything is not as the fast case has it (a wrong tensor, no
// workspace, a sequence that is no list or tuple).  The caller then takes the same steps
// in Python, which says what is wrong.  Nothing is kept between calls but what setup()
// gave, and no exception leaves a function.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "oscar.h"

namespace {

constexpr int MAX_REQ = 256, HEAD_DIM = 128;
constexpr c10::ScalarType BF16 = c10::kBFloat16, F32 = c10::kFloat, I32 = c10::kInt, U8 = c10::kByte;

using append16_fn = oscar_status (*)(void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t,
                                    int32_t, int32_t, const oscar_rope*, const uint16_t*, int64_t, const uint16_t*,
                                    int64_t, const uint16_t*, int64_t, uint16_t*, int32_t*, void*);
using append4_fn = oscar_status (*)(void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t,
                                   int32_t, int32_t, int32_t, const oscar_rope*, const uint16_t*, int64_t,
                                   const uint16_t*, int64_t, const uint16_t*, int64_t, uint16_t*, int32_t*, void*);
using read4_fn = oscar_status (*)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                 int32_t, int32_t, int32_t, void*, void*, int32_t, int32_t*, void*);
using attend16_fn = oscar_status (*)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                    int32_t, int32_t, int32_t, int32_t, int32_t, float, const uint16_t*, int64_t, void*,
                                    int32_t, float*, int32_t*, void*, size_t, void*);
using attend4_fn = oscar_status (*)(const void*, int64_t, const int32_t*, int32_t, const int32_t*, const int32_t*,
                                   int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, float, const uint16_t*,
                                   int64_t, void*, int32_t, float*, int32_t*, void*, size_t, void*);

struct {
  append16_fn append16;
  append4_fn append4;
  read4_fn read4;
  attend16_fn attend16;
  attend4_fn attend4;
} g;

// A tensor argument that is as it should be, or null.
const at::Tensor* tensor(PyObject* o, c10::ScalarType type, int device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || t.scalar_type() != type || !t.is_cuda() || t.get_device() != device) return nullptr;
  return &t;
}
// dense, too, and of the given shape (none: any; a negative extent: any)
const at::Tensor* dense(PyObject* o, c10::ScalarType type, int device, std::initializer_list<int64_t> shape = {}) {
  const at::Tensor* t = tensor(o, type, device);
  if (!t || !t->is_contiguous()) return nullptr;
  if (shape.size()) {
    const c10::IntArrayRef have = t->sizes();
    if (have.size() != shape.size()) return nullptr;
    const int64_t* want = shape.begin();
    for (size_t i = 0; i < have.size(); ++i)
      if (have[i] != want[i] && want[i] >= 0) return nullptr;
  }
  return t;
}
// bf16 [rows][heads][128] whose heads lie densely; heads < 0: any.  stride: from token to token
const at::Tensor* heads_of(PyObject* o, int device, int64_t rows, int64_t heads, int64_t* stride) {
  const at::Tensor* t = tensor(o, BF16, device);
  if (!t || t->dim() != 3) return nullptr;
  const c10::IntArrayRef n = t->sizes(), s = t->strides();
  if (n[0] != rows || (heads >= 0 && n[1] != heads) || n[2] != HEAD_DIM || s[2] != 1 || (s[1] != HEAD_DIM && n[1] > 1))
    return nullptr;
  *stride = rows > 1 ? s[0] : n[1] * HEAD_DIM;
  return t;
}
const at::Tensor* error_word(PyObject* o, int device) {
  const at::Tensor* t = dense(o, I32, device);
  return t && t->numel() > 0 ? t : nullptr;
}
template <typename T>
T* at_ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
const at::Tensor* pool_of(PyObject* kv, long group, int device, int64_t hkv) {
  if (group == 0) return dense(kv, BF16, device, {-1, hkv, 2, 64, HEAD_DIM});
  return group == 128 || group == 64 ? dense(kv, U8, device, {-1, hkv, group == 128 ? 8704 : 9216}) : nullptr;
}

// host ints of a list or tuple of n, not negative; their sum, or -1
int64_t counts(PyObject* o, Py_ssize_t n, int32_t* out) {
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

// the call's stream: torch's current one on the current device, where none is given
bool context(PyObject* stream, int* device, void** raw) {
  if (stream != Py_None || !g.append16) return false;
  const c10::cuda::CUDAStream s = c10::cuda::getCurrentCUDAStream();
  *device = s.device_index();
  *raw = s.stream();
  return true;
}

long group_of(PyObject* o) {   // -1: no int
  const long v = PyLong_AsLong(o);
  if (v == -1) PyErr_Clear();
  return v;
}

Py_ssize_t requests(PyObject* lens) {
  if (!(PyList_Check(lens) || PyTuple_Check(lens))) return 0;
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(lens);
  return n <= MAX_REQ ? n : 0;
}

// append(group, kv, page_table, lens, k, v, rope, q, q_out, new_lens, interleaved, error, stream): status, or -1
int append(PyObject* const* a, Py_ssize_t count) {
  int32_t lens[MAX_REQ], news[MAX_REQ];
  int device;
  void* stream;
  if (count != 13 || !context(a[12], &device, &stream)) return -1;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || counts(a[3], n, lens) < 0) return -1;
  int64_t rows = n;
  if (a[9] != Py_None && (rows = counts(a[9], n, news)) < 0) return -1;
  int64_t ks, vs, qs = 0, hq = 0;
  const at::Tensor *k = heads_of(a[4], device, rows, -1, &ks), *q = nullptr, *q_out = nullptr, *err = nullptr;
  if (!k) return -1;
  const int64_t hkv = k->size(1);
  const at::Tensor *v = heads_of(a[5], device, rows, hkv, &vs), *kv = pool_of(a[1], group, device, hkv),
                   *table = dense(a[2], I32, device, {n, -1});
  if (!v || !kv || !table) return -1;
  if (a[7] != Py_None && a[8] != Py_None) {
    if (!(q = heads_of(a[7], device, rows, -1, &qs))) return -1;
    hq = q->size(1);
    if (!(q_out = dense(a[8], BF16, device, {rows, hq, HEAD_DIM}))) return -1;
  } else if (a[7] != a[8]) {
    return -1;
  }
  oscar_rope r;
  const oscar_rope* rope = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor* t = dense(a[6], F32, device, {-1, -1});
    const int inter = PyObject_IsTrue(a[10]);
    if (!t || t->size(0) > INT32_MAX || t->size(1) > INT32_MAX || inter < 0) return -1;
    r = {at_ptr<const float>(t), static_cast<int32_t>(t->size(0)), static_cast<int32_t>(t->size(1)), inter};
    rope = &r;
  }
  if (a[11] != Py_None && !(err = error_word(a[11], device))) return -1;
  if (table->size(1) > INT32_MAX || hkv > INT32_MAX || hq > INT32_MAX) return -1;
  if (rows == 0) return OSCAR_OK;
  const int32_t* nl = a[9] == Py_None ? nullptr : news;
  const int64_t pages = kv->size(0);
  const int32_t max_pages = static_cast<int32_t>(table->size(1));
  void* pool = kv->data_ptr();
  const auto* pt = at_ptr<const int32_t>(table);
  const auto *qp = at_ptr<const uint16_t>(q), *kp = at_ptr<const uint16_t>(k), *vp = at_ptr<const uint16_t>(v);
  auto* qo = at_ptr<uint16_t>(q_out);
  auto* ep = at_ptr<int32_t>(err);
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  if (group == 0)
    st = g.append16(pool, pages, pt, max_pages, lens, nl, static_cast<int32_t>(n), static_cast<int32_t>(hq),
                    static_cast<int32_t>(hkv), rope, qp, qs, kp, ks, vp, vs, qo, ep, stream);
  else
    st = g.append4(pool, pages, pt, max_pages, lens, nl, static_cast<int32_t>(n), static_cast<int32_t>(hq),
                   static_cast<int32_t>(hkv), static_cast<int32_t>(group), rope, qp, qs, kp, ks, vp, vs, qo, ep, stream);
  Py_END_ALLOW_THREADS
  return st;
}

// read(group, kv, page_table, starts, counts, k_out, v_out, error, stream)
int read(PyObject* const* a, Py_ssize_t count) {
  int32_t starts[MAX_REQ], cnt[MAX_REQ];
  int device;
  void* stream;
  if (count != 9 || !context(a[8], &device, &stream)) return -1;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || group == 0 || counts(a[3], n, starts) < 0) return -1;
  const int64_t rows = counts(a[4], n, cnt);
  if (rows < 0) return -1;
  const bool f32 = tensor(a[5], F32, device) != nullptr;
  const c10::ScalarType kind = f32 ? F32 : BF16;
  const at::Tensor *ko = dense(a[5], kind, device, {rows, -1, HEAD_DIM}), *err = nullptr;
  if (!ko) return -1;
  const int64_t hkv = ko->size(1);
  const at::Tensor *vo = dense(a[6], kind, device, {rows, hkv, HEAD_DIM}), *kv = pool_of(a[1], group, device, hkv),
                   *table = dense(a[2], I32, device, {n, -1});
  if (!vo || !kv || !table || table->size(1) > INT32_MAX || hkv > INT32_MAX) return -1;
  if (a[7] != Py_None && !(err = error_word(a[7], device))) return -1;
  if (rows == 0) return OSCAR_OK;
  const int64_t pages = kv->size(0);
  const int32_t max_pages = static_cast<int32_t>(table->size(1));
  const void* pool = kv->data_ptr();
  const auto* pt = at_ptr<const int32_t>(table);
  void *kp = ko->data_ptr(), *vp = vo->data_ptr();
  auto* ep = at_ptr<int32_t>(err);
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  st = g.read4(pool, pages, pt, max_pages, starts, cnt, static_cast<int32_t>(n), static_cast<int32_t>(hkv),
               static_cast<int32_t>(group), kp, vp, f32 ? OSCAR_F32 : OSCAR_BF16, ep, stream);
  Py_END_ALLOW_THREADS
  return st;
}

// attend(group, kv, page_table, lens, q, out, num_kv_heads, window, sinks, q_lens, scale, lse, workspace, error, stream)
int attend(PyObject* const* a, Py_ssize_t count) {
  int32_t lens[MAX_REQ], ql[MAX_REQ];
  int device;
  void* stream;
  if (count != 15 || a[12] == Py_None || !context(a[14], &device, &stream)) return -1;
  const long group = group_of(a[0]);
  const Py_ssize_t n = requests(a[3]);
  if (n == 0 || counts(a[3], n, lens) < 0) return -1;
  int64_t rows = n;
  if (a[9] != Py_None && (rows = counts(a[9], n, ql)) < 0) return -1;
  const long long hkv = PyLong_AsLongLong(a[6]), window = PyLong_AsLongLong(a[7]), sinks = PyLong_AsLongLong(a[8]);
  const double scale = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred() || hkv < 1 || hkv > INT32_MAX || window < INT32_MIN || window > INT32_MAX || sinks < 0 ||
      sinks > INT32_MAX)
    return -1;
  int64_t qs;
  const at::Tensor* q = heads_of(a[4], device, rows, -1, &qs);
  if (!q) return -1;
  const int64_t hq = q->size(1);
  const bool f32 = tensor(a[5], F32, device) != nullptr;
  const at::Tensor *out = dense(a[5], f32 ? F32 : BF16, device, {rows, hq, HEAD_DIM}),
                   *kv = pool_of(a[1], group, device, hkv), *table = dense(a[2], I32, device, {n, -1}),
                   *ws = dense(a[12], U8, device, {-1}), *lse = nullptr, *err = nullptr;
  if (!out || !kv || !table || !ws || table->size(1) > INT32_MAX || hq > INT32_MAX) return -1;
  if (a[11] != Py_None && !(lse = dense(a[11], F32, device, {rows, hq}))) return -1;
  if (a[13] != Py_None && !(err = error_word(a[13], device))) return -1;
  if (rows == 0) return OSCAR_OK;
  const int32_t* qn = a[9] == Py_None ? nullptr : ql;
  const int64_t pages = kv->size(0);
  const int32_t max_pages = static_cast<int32_t>(table->size(1)), kind = f32 ? OSCAR_F32 : OSCAR_BF16;
  const void* pool = kv->data_ptr();
  const auto* pt = at_ptr<const int32_t>(table);
  const auto* qp = at_ptr<const uint16_t>(q);
  void *op = out->data_ptr(), *wp = ws->data_ptr();
  auto* lp = at_ptr<float>(lse);
  auto* ep = at_ptr<int32_t>(err);
  const size_t ws_bytes = static_cast<size_t>(ws->size(0));
  oscar_status st;
  Py_BEGIN_ALLOW_THREADS
  if (group == 0)
    st = g.attend16(pool, pages, pt, max_pages, lens, qn, static_cast<int32_t>(n), static_cast<int32_t>(hq),
                    static_cast<int32_t>(hkv), static_cast<int32_t>(window), static_cast<int32_t>(sinks),
                    static_cast<float>(scale), qp, qs, op, kind, lp, ep, wp, ws_bytes, stream);
  else
    st = g.attend4(pool, pages, pt, max_pages, lens, qn, static_cast<int32_t>(n), static_cast<int32_t>(hq),
                   static_cast<int32_t>(hkv), static_cast<int32_t>(group), static_cast<int32_t>(window),
                   static_cast<int32_t>(sinks), static_cast<float>(scale), qp, qs, op, kind, lp, ep, wp, ws_bytes,
                   stream);
  Py_END_ALLOW_THREADS
  return st;
}

template <int (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t count) {
  int st = -1;
  try {
    st = F(a, count);
  } catch (...) {   // a tensor without memory, no device
  }
  if (st >= 0) return PyLong_FromLong(st);
  PyErr_Clear();
  Py_RETURN_NONE;
}

// setup((five function addresses))
PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long at[5];
  if (!PyArg_ParseTuple(args, "(KKKKK)", &at[0], &at[1], &at[2], &at[3], &at[4])) return nullptr;
  g = {reinterpret_cast<append16_fn>(at[0]), reinterpret_cast<append4_fn>(at[1]), reinterpret_cast<read4_fn>(at[2]),
       reinterpret_cast<attend16_fn>(at[3]), reinterpret_cast<attend4_fn>(at[4])};
  Py_RETURN_NONE;
}

template <int (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F>));
}
PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                         {"append", fast<append>(), METH_FASTCALL, nullptr},
                         {"read", fast<read>(), METH_FASTCALL, nullptr},
                         {"attend", fast<attend>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_oscar_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__oscar_calls(void) { return PyModule_Create(&module); }
