// The checks and the call of the short operators, for Python.
//
// The wrappers in binding.py check every tensor and hand raw pointers to the C
// ABI through ctypes; for kernels of a few microseconds that costs more time
// than the kernel (measured on B200: 6 to 10 us a call, 3 to 4 of them the
// checks).  These functions make the same checks on the tensors themselves.  A call
// that passes them is made at once and its status returned; for anything else
// they return None without a call, and the wrapper's own checks say what is
// wrong.  Nothing is kept from one call for the next.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "../../include/mla.h"

namespace {

using at::ScalarType;

decltype(&mla_rope) f_rope;
decltype(&mla_plan_pages_capped) f_plan_pages;
decltype(&mla_cache_write_paged_step) f_write;
decltype(&mla_cache_write_fp8_paged) f_write8;
decltype(&mla_decode_fp8_paged) f_decode8;

constexpr int64_t kPageRows = 64;

// One call's checks: after the first that fails, ok stays false.
struct Call {
  bool ok = true;
  int dev = -1;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda()) {
      ok = false;
      return nullptr;
    }
    const int d = t.get_device();
    if (dev < 0) {
      // A call on another device than the current one takes the wrapper's way.
      dev = d;
      ok = ok && d == c10::cuda::current_device();
    }
    ok = ok && d == dev;
    return &t;
  }
  // Address of a contiguous tensor of this type and shape.
  void* arg(PyObject* o, ScalarType type, std::initializer_list<int64_t> shape) {
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    ok = t->scalar_type() == type && t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
    return ok ? t->data_ptr() : nullptr;
  }
  void* optional(PyObject* o, ScalarType type, std::initializer_list<int64_t> shape) {
    return o == Py_None ? nullptr : arg(o, type, shape);
  }
  // Rows [T, width] with unit inner stride; any row stride.
  void* rows(PyObject* o, ScalarType type, int64_t width, int64_t* T, int64_t* stride) {
    const at::Tensor* t = tensor(o);
    if (!ok) return nullptr;
    ok = t->scalar_type() == type && t->dim() == 2 && t->size(1) == width && t->stride(1) == 1;
    if (!ok) return nullptr;
    *T = t->size(0);
    *stride = *T > 1 ? t->stride(0) : width;
    return t->data_ptr();
  }
  int64_t size(PyObject* o, int64_t dim) {
    const at::Tensor* t = tensor(o);
    if (!ok || t->dim() <= dim) {
      ok = false;
      return 0;
    }
    return t->size(dim);
  }
  // A rope table, read through its buffer.
  const mla_rope_table* table(PyObject* o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) {
      PyErr_Clear();
      ok = false;
      return nullptr;
    }
    const auto* t = static_cast<const mla_rope_table*>(b.buf);
    ok = ok && b.len == Py_ssize_t(sizeof(mla_rope_table));
    PyBuffer_Release(&b);      // the caller's reference keeps the memory
    return ok ? t : nullptr;
  }
  const mla_dims* dims(PyObject* o) {
    const void* p = PyLong_AsVoidPtr(o);
    if (!p) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<const mla_dims*>(p);
  }
  int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return float(v);
  }
  bool fits32(int64_t v) { return ok = ok && v >= 0 && v <= INT32_MAX; }
  void* stream() { return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream(); }
};

PyObject* status(int st) { return PyLong_FromLong(st); }

#define MLA_SLOW_UNLESS(cond) \
  if (!(cond)) Py_RETURN_NONE

ScalarType scalar(const mla_dims* d) {
  return d->dtype == MLA_BF16 ? ScalarType::BFloat16 : ScalarType::Float;
}

// rope(table, x, pos, out, transpose)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  MLA_SLOW_UNLESS(n == 5);
  const mla_rope_table* tab = c.table(a[0]);
  const at::Tensor* x = c.ok ? c.tensor(a[1]) : nullptr;
  const at::Tensor* y = c.ok ? c.tensor(a[3]) : nullptr;
  MLA_SLOW_UNLESS(c.ok);
  const int64_t nd = x->dim();
  const ScalarType type = x->scalar_type();
  MLA_SLOW_UNLESS((nd == 2 || nd == 3) && (type == ScalarType::BFloat16 || type == ScalarType::Float) &&
                  y->scalar_type() == type && y->sizes() == x->sizes() &&
                  x->size(nd - 1) == tab->d_r && x->stride(nd - 1) == 1 && y->stride(nd - 1) == 1);
  const int64_t T = x->size(0), H = nd == 3 ? x->size(1) : 1;
  const void* pos = c.arg(a[2], ScalarType::Int, {T});
  const int transpose = PyObject_IsTrue(a[4]);
  if (transpose < 0) PyErr_Clear();
  MLA_SLOW_UNLESS(c.ok && transpose >= 0 && H > 0 && c.fits32(H));
  return status(f_rope(type == ScalarType::BFloat16 ? MLA_BF16 : MLA_F32, tab, T, int32_t(H),
                       x->data_ptr(), x->stride(0), nd == 3 ? x->stride(1) : 0,
                       static_cast<const int32_t*>(pos), y->data_ptr(), y->stride(0),
                       nd == 3 ? y->stride(1) : 0, transpose, c.stream()));
}

// plan_pages(seqlens, new_lens, block_table, free_pages, free_count, num_pages, query_start,
//            positions, slots, seqlens_out, free_count_out, workspace, token_request, capacity)
PyObject* plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  MLA_SLOW_UNLESS(n == 14);
  const ScalarType i32 = ScalarType::Int;
  const int64_t B = c.size(a[0], 0), blocks = c.size(a[2], 1), F = c.size(a[3], 0),
                T = c.size(a[7], 0);
  MLA_SLOW_UNLESS(c.ok && c.fits32(B) && c.fits32(blocks) && c.fits32(F) && c.fits32(T));
  const void* seq = c.arg(a[0], i32, {B});
  const void* add = c.arg(a[1], i32, {B});
  void* table = c.arg(a[2], i32, {B, blocks});
  const void* free_pages = c.arg(a[3], i32, {F});
  const void* count = c.arg(a[4], i32, {1});
  const int64_t pages = c.integer(a[5]);
  void* qs = c.arg(a[6], i32, {B + 1});
  void* pos = c.arg(a[7], i32, {T});
  void* slots = c.arg(a[8], ScalarType::Long, {T});
  void* seq_out = c.arg(a[9], i32, {B});
  void* count_out = c.arg(a[10], i32, {1});
  const at::Tensor* ws = c.ok ? c.tensor(a[11]) : nullptr;
  void* request = c.ok ? c.optional(a[12], i32, {T}) : nullptr;
  const int64_t capacity = a[13] == Py_None ? blocks * kPageRows : c.integer(a[13]);
  MLA_SLOW_UNLESS(c.ok && ws->is_contiguous());
  return status(f_plan_pages(
      int32_t(B), static_cast<const int32_t*>(seq), static_cast<const int32_t*>(add),
      static_cast<int32_t*>(table), int32_t(blocks), capacity,
      static_cast<const int32_t*>(free_pages), int32_t(F), static_cast<const int32_t*>(count), pages, int32_t(T),
      static_cast<int32_t*>(qs), static_cast<int32_t*>(pos), static_cast<int64_t*>(slots),
      static_cast<int32_t*>(request), static_cast<int32_t*>(seq_out),
      static_cast<int32_t*>(count_out), ws->data_ptr(), ws->nbytes(), c.stream()));
}

// cache_write_paged(dims, x, gamma, positions, slots, cache_pool, table, eps, planned)
PyObject* cache_write_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  MLA_SLOW_UNLESS(n == 9);
  const mla_dims* d = c.dims(a[0]);
  MLA_SLOW_UNLESS(c.ok);
  const int64_t R = int64_t(d->d_c) + d->d_r;
  int64_t T = 0, stride = 0;
  const void* x = c.rows(a[1], scalar(d), R, &T, &stride);
  MLA_SLOW_UNLESS(c.ok && c.fits32(T));
  const void* gamma = c.optional(a[2], ScalarType::Float, {d->d_c});
  const void* pos = c.optional(a[3], ScalarType::Int, {T});
  const void* slots = c.arg(a[4], ScalarType::Long, {T});
  const int64_t pages = c.size(a[5], 0);
  void* pool = c.arg(a[5], scalar(d), {pages, kPageRows, R});
  const mla_rope_table* tab = a[6] == Py_None ? nullptr : c.table(a[6]);
  const float eps = c.real(a[7]);
  const void* planned = c.ok ? c.optional(a[8], ScalarType::Int, {1}) : nullptr;
  MLA_SLOW_UNLESS(c.ok);
  return status(f_write(d, int32_t(T), x, stride, static_cast<const float*>(gamma), eps, tab,
                        static_cast<const int32_t*>(pos), static_cast<const int64_t*>(slots),
                        static_cast<const int32_t*>(planned), pool, pages, c.stream()));
}

// cache_write_fp8_paged(dims, x, gamma, query_start, seqlens, block_table, cache_pool,
//                       page_scales, table, eps)
PyObject* cache_write_fp8_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  MLA_SLOW_UNLESS(n == 10);
  const mla_dims* d = c.dims(a[0]);
  MLA_SLOW_UNLESS(c.ok);
  const int64_t B = d->B;
  int64_t T = 0, stride = 0;
  const void* x = c.rows(a[1], scalar(d), int64_t(d->d_c) + d->d_r, &T, &stride);
  MLA_SLOW_UNLESS(c.ok && c.fits32(T));
  const void* gamma = c.optional(a[2], ScalarType::Float, {d->d_c});
  const void* qs = c.arg(a[3], ScalarType::Int, {B + 1});
  const void* seq = c.arg(a[4], ScalarType::Int, {B});
  const int64_t blocks = c.size(a[5], 1), pages = c.size(a[6], 0);
  const void* table = c.arg(a[5], ScalarType::Int, {B, blocks});
  void* pool = c.arg(a[6], ScalarType::Byte, {pages, kPageRows, int64_t(d->d_c) + 2 * d->d_r});
  void* scales = c.arg(a[7], ScalarType::Float, {pages});
  const mla_rope_table* tab = a[8] == Py_None ? nullptr : c.table(a[8]);
  const float eps = c.real(a[9]);
  MLA_SLOW_UNLESS(c.ok && c.fits32(blocks));
  return status(f_write8(d, int32_t(T), x, stride, static_cast<const float*>(gamma), eps, tab,
                         static_cast<const int32_t*>(qs), static_cast<const int32_t*>(seq),
                         static_cast<const int32_t*>(table), int32_t(blocks), pool,
                         static_cast<float*>(scales), pages, c.stream()));
}

// decode_fp8_paged(dims, q_cat, cache_pool, page_scales, block_table, seqlens, softmax_scale,
//                  workspace, num_splits) -> the splits used, or minus the status
PyObject* decode_fp8_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Call c;
  MLA_SLOW_UNLESS(n == 9);
  const mla_dims* d = c.dims(a[0]);
  MLA_SLOW_UNLESS(c.ok);
  const int64_t B = d->B;
  const void* q = c.arg(a[1], scalar(d), {B, d->H, int64_t(d->d_c) + d->d_r});
  const int64_t pages = c.ok ? c.size(a[2], 0) : 0, blocks = c.ok ? c.size(a[4], 1) : 0;
  MLA_SLOW_UNLESS(c.ok && c.fits32(blocks));
  const void* pool = c.arg(a[2], ScalarType::Byte, {pages, kPageRows, int64_t(d->d_c) + 2 * d->d_r});
  const void* scales = c.arg(a[3], ScalarType::Float, {pages});
  const void* table = c.arg(a[4], ScalarType::Int, {B, blocks});
  const void* seq = c.arg(a[5], ScalarType::Int, {B});
  const float scale = c.real(a[6]);
  const at::Tensor* ws = c.ok ? c.tensor(a[7]) : nullptr;
  const int64_t splits = c.integer(a[8]);
  MLA_SLOW_UNLESS(c.ok && ws->is_contiguous() && c.fits32(splits));
  int used = 0;
  const int st =
      f_decode8(d, q, pool, static_cast<const float*>(scales), pages,
                static_cast<const int32_t*>(table), int32_t(blocks),
                static_cast<const int32_t*>(seq), scale, int(splits), ws->data_ptr(), ws->nbytes(),
                &used, c.stream());
  return PyLong_FromLong(st ? -st : used);
}

// init(addresses of the library's functions, in the order below)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "init takes 5 addresses");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
  f_plan_pages = reinterpret_cast<decltype(f_plan_pages)>(p[1]);
  f_write = reinterpret_cast<decltype(f_write)>(p[2]);
  f_write8 = reinterpret_cast<decltype(f_write8)>(p[3]);
  f_decode8 = reinterpret_cast<decltype(f_decode8)>(p[4]);
  Py_RETURN_NONE;
}

// No C++ exception reaches Python: a check that throws is a call for the wrapper.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

#define MLA_METHOD(f) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&init)), METH_FASTCALL, nullptr},
    MLA_METHOD(rope),
    MLA_METHOD(plan_pages),
    MLA_METHOD(cache_write_paged),
    MLA_METHOD(cache_write_fp8_paged),
    MLA_METHOD(decode_fp8_paged),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods,
                      nullptr,               nullptr,  nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
