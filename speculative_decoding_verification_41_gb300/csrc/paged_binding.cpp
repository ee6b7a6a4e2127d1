// paged_binding.cpp -- the Python module behind paged.py's usual calls: checks of
// the arguments and marshalling for libdspark's paged-cache entry points
// (include/dspark_paged.h), as paged.py states them, without the interpreter.
//
// The calls take a few microseconds on the GPU, and attribute by attribute the
// checks and a ctypes call took 6 to 8 on the host. A call whose arguments do not
// pass here returns None, and paged.py's own statement of the checks then says
// what is wrong (or handles it: other devices, outputs not yet allocated).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dspark_paged.h"

namespace {

decltype(&dspark_pages_reserve) g_reserve;
decltype(&dspark_pages_release) g_release;
decltype(&dspark_kv_append) g_append;
decltype(&dspark_paged_attention) g_attention;

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}
// a contiguous tensor of this type on CUDA device `dev`
bool plain(const at::Tensor* t, at::ScalarType type, int dev) {
  return t && t->scalar_type() == type && t->is_cuda() && t->get_device() == dev &&
         t->is_contiguous();
}
// ... of this shape
bool plain(const at::Tensor* t, at::ScalarType type, int dev, at::IntArrayRef shape) {
  return plain(t, type, dev) && t->sizes() == shape;
}
template <typename T>
T* data(const at::Tensor* t) {
  return static_cast<T*>(t->data_ptr());
}
bool whole(PyObject* o, int64_t& v) {
  v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool small(PyObject* o, int32_t& v) {
  int64_t w;
  if (!whole(o, w) || w < INT32_MIN || w > INT32_MAX) return false;
  v = static_cast<int32_t>(w);
  return true;
}
// rows of a block table [B][width]
bool table(const at::Tensor* t, int dev, int64_t B, int64_t& stride, int32_t& width) {
  if (!t || t->scalar_type() != at::kInt || !t->is_cuda() || t->get_device() != dev ||
      t->dim() != 2 || t->size(0) != B || t->size(1) > INT32_MAX ||
      (t->stride(1) != 1 && t->size(1) > 1))
    return false;
  width = static_cast<int32_t>(t->size(1));
  stride = B > 1 ? t->stride(0) : width;
  return true;
}
// A call of the current device: others go the long way.
bool here(int dev) { return c10::cuda::current_device() == dev; }
bool stream_of(PyObject* o, int dev, CUstream_st*& s) {
  if (o == Py_None) {
    s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return true;
  }
  int64_t v;
  if (!whole(o, v)) return false;
  s = reinterpret_cast<CUstream_st*>(v);
  return true;
}
bool element(at::ScalarType t, int32_t& dtype) {
  if (t == at::kBFloat16)
    dtype = DSPARK_BF16;
  else if (t == at::kHalf)
    dtype = DSPARK_F16;
  else
    return false;
  return true;
}
struct Cache {
  int64_t pages, page_size, heads, D;
  int64_t page, token, head;
  int32_t dtype;
};
bool cache(const at::Tensor* k, const at::Tensor* v, int dev, Cache& c) {
  if (!k || !v || !k->is_cuda() || !v->is_cuda() || v->get_device() != dev || k->dim() != 4 ||
      k->stride(3) != 1 || k->sizes() != v->sizes() || k->strides() != v->strides() ||
      k->scalar_type() != v->scalar_type() || !element(k->scalar_type(), c.dtype))
    return false;
  c.pages = k->size(0), c.page_size = k->size(1), c.heads = k->size(2), c.D = k->size(3);
  c.page = k->stride(0), c.token = k->stride(1), c.head = k->stride(2);
  return c.pages <= INT32_MAX && c.page_size <= INT32_MAX && c.heads <= INT32_MAX &&
         c.D <= INT32_MAX;
}

PyObject* done(int rc) { return PyLong_FromLong(rc); }

#define REFUSE_UNLESS(x) \
  do {                   \
    if (!(x)) Py_RETURN_NONE; \
  } while (0)

// reserve(context_len, new_len, block_table, free_pages, free_count, page_size, max_tokens,
//         extra, context_out, row_off, draft_off, slot_map, positions, free_out, status, stream)
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 16 && g_reserve);
  const at::Tensor* t[15] = {};
  for (int i : {0, 1, 2, 3, 4, 8, 9, 10, 11, 12, 13, 14}) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[0]->is_cuda());
  const int dev = t[0]->get_device();
  const int64_t B = t[0]->numel();
  int32_t page_size, max_tokens, extra, width;
  int64_t stride;
  CUstream_st* s;
  REFUSE_UNLESS(B <= INT32_MAX && small(a[5], page_size) && small(a[6], max_tokens) &&
                small(a[7], extra) && max_tokens >= 0);
  REFUSE_UNLESS(plain(t[0], at::kInt, dev, B) && plain(t[1], at::kInt, dev, B) &&
                table(t[2], dev, B, stride, width) && plain(t[3], at::kInt, dev) &&
                t[3]->numel() <= INT32_MAX && plain(t[4], at::kInt, dev, 1) &&
                plain(t[8], at::kInt, dev, B) && plain(t[9], at::kLong, dev, B + 1) &&
                plain(t[10], at::kLong, dev, B + 1) && plain(t[11], at::kInt, dev, max_tokens) &&
                plain(t[12], at::kInt, dev, max_tokens) && plain(t[13], at::kInt, dev, 1) &&
                plain(t[14], at::kInt, dev, 1) && here(dev) && stream_of(a[15], dev, s));
  return done(g_reserve(data<int32_t>(t[0]), data<int32_t>(t[1]), extra, static_cast<int32_t>(B),
                        page_size, static_cast<int32_t>(t[3]->numel()), data<int32_t>(t[2]),
                        stride, width, data<int32_t>(t[3]), data<int32_t>(t[4]), max_tokens,
                        data<int32_t>(t[8]), data<int64_t>(t[9]), data<int64_t>(t[10]),
                        data<int32_t>(t[11]), data<int32_t>(t[12]), data<int32_t>(t[13]),
                        data<int32_t>(t[14]), s));
}

// release(context_len, reserved_len, kept_len, block_table, free_pages, free_count, page_size,
//         extra, context_out, free_out, status, stream)
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 12 && g_release);
  const at::Tensor* t[11] = {};
  for (int i : {0, 1, 2, 3, 4, 5, 8, 9, 10}) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[0]->is_cuda());
  const int dev = t[0]->get_device();
  const int64_t B = t[0]->numel();
  int32_t page_size, extra, width;
  int64_t stride;
  CUstream_st* s;
  REFUSE_UNLESS(B <= INT32_MAX && small(a[6], page_size) && small(a[7], extra));
  REFUSE_UNLESS(plain(t[0], at::kInt, dev, B) && plain(t[1], at::kInt, dev, B) &&
                plain(t[2], at::kInt, dev, B) && table(t[3], dev, B, stride, width) &&
                plain(t[4], at::kInt, dev) && t[4]->numel() <= INT32_MAX &&
                plain(t[5], at::kInt, dev, 1) && plain(t[8], at::kInt, dev, B) &&
                plain(t[9], at::kInt, dev, 1) && plain(t[10], at::kInt, dev, 1) && here(dev) &&
                stream_of(a[11], dev, s));
  return done(g_release(data<int32_t>(t[0]), data<int32_t>(t[1]), data<int32_t>(t[2]), extra,
                        static_cast<int32_t>(B), page_size, static_cast<int32_t>(t[4]->numel()),
                        data<int32_t>(t[3]), stride, width, data<int32_t>(t[4]),
                        data<int32_t>(t[5]), data<int32_t>(t[8]), data<int32_t>(t[9]),
                        data<int32_t>(t[10]), s));
}

// append(k, v, slot_map, k_cache, v_cache, status, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 7 && g_append);
  const at::Tensor* t[6];
  for (int i = 0; i < 6; ++i) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[1] && t[3] && t[3]->is_cuda());
  const int dev = t[3]->get_device();
  Cache c;
  CUstream_st* s;
  REFUSE_UNLESS(cache(t[3], t[4], dev, c));
  REFUSE_UNLESS(t[0]->is_cuda() && t[1]->is_cuda() && t[0]->get_device() == dev &&
                t[1]->get_device() == dev && t[0]->dim() == 3 && t[0]->stride(2) == 1 &&
                t[0]->size(0) <= INT32_MAX && t[0]->size(1) == c.heads && t[0]->size(2) == c.D &&
                t[0]->sizes() == t[1]->sizes() && t[0]->strides() == t[1]->strides() &&
                t[0]->scalar_type() == t[3]->scalar_type() &&
                t[1]->scalar_type() == t[3]->scalar_type() && plain(t[2], at::kInt, dev) &&
                t[2]->numel() >= t[0]->size(0) && plain(t[5], at::kInt, dev, 1) && here(dev) &&
                stream_of(a[6], dev, s));
  return done(g_append(t[0]->data_ptr(), t[1]->data_ptr(), t[0]->stride(0), t[0]->stride(1),
                       data<int32_t>(t[2]), static_cast<int32_t>(t[0]->size(0)),
                       static_cast<int32_t>(c.heads), static_cast<int32_t>(c.D), c.dtype,
                       t[3]->data_ptr(), t[4]->data_ptr(), c.page, c.token, c.head,
                       static_cast<int32_t>(c.page_size), static_cast<int32_t>(c.pages),
                       data<int32_t>(t[5]), s));
}

// attention(q, k_cache, v_cache, block_table, context_len, row_off, scale, max_new, window, out,
//           lse or None, status, workspace, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 14 && g_attention);
  const at::Tensor* t[13] = {};
  for (int i : {0, 1, 2, 3, 4, 5, 9, 10, 11, 12}) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[1] && t[4] && t[9] && t[12] && t[1]->is_cuda());
  const int dev = t[1]->get_device();
  Cache c;
  CUstream_st* s;
  REFUSE_UNLESS(cache(t[1], t[2], dev, c));
  const at::Tensor& q = *t[0];
  const int64_t B = t[4]->numel();
  int64_t stride;
  int32_t width, max_new, window;
  const double scale = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  REFUSE_UNLESS(small(a[7], max_new) && small(a[8], window) && max_new >= 1);
  REFUSE_UNLESS(q.is_cuda() && q.get_device() == dev && q.dim() == 3 && q.stride(2) == 1 &&
                q.size(2) == c.D && q.scalar_type() == t[1]->scalar_type() &&
                q.size(0) <= INT32_MAX && q.size(1) <= INT32_MAX && c.heads >= 1 &&
                q.size(1) >= 1 && q.size(1) % c.heads == 0);
  REFUSE_UNLESS(B <= INT32_MAX && plain(t[4], at::kInt, dev, B) &&
                plain(t[5], at::kLong, dev, B + 1) && table(t[3], dev, B, stride, width) &&
                plain(t[9], q.scalar_type(), dev, q.sizes()) &&
                (a[10] == Py_None || plain(t[10], at::kFloat, dev, {q.size(0), q.size(1)})) &&
                plain(t[11], at::kInt, dev, 1) && plain(t[12], at::kByte, dev) && here(dev) &&
                stream_of(a[13], dev, s));
  return done(g_attention(
      q.data_ptr(), q.stride(0), q.stride(1), t[1]->data_ptr(), t[2]->data_ptr(), c.page, c.token,
      c.head, static_cast<int32_t>(c.page_size), static_cast<int32_t>(c.pages),
      data<int32_t>(t[3]), stride, width, data<int32_t>(t[4]), data<int64_t>(t[5]),
      static_cast<int32_t>(B), static_cast<int32_t>(q.size(0)), static_cast<int32_t>(q.size(1)),
      static_cast<int32_t>(c.heads), static_cast<int32_t>(c.D), max_new,
      static_cast<float>(scale), window, c.dtype, t[9]->data_ptr(),
      a[10] == Py_None ? nullptr : data<float>(t[10]), data<int32_t>(t[11]), t[12]->data_ptr(),
      static_cast<size_t>(t[12]->numel()), s));
}

// C++ exceptions (a CUDA error in torch's own calls) become Python's.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(reserve, release, append, attention): addresses of libdspark's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t f[4];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i)
    if (!whole(a[i], f[i])) {
      PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
      return nullptr;
    }
  g_reserve = reinterpret_cast<decltype(g_reserve)>(f[0]);
  g_release = reinterpret_cast<decltype(g_release)>(f[1]);
  g_append = reinterpret_cast<decltype(g_append)>(f[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[3]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"reserve", fast(guarded<reserve>), METH_FASTCALL, nullptr},
    {"release", fast(guarded<release>), METH_FASTCALL, nullptr},
    {"append", fast(guarded<append>), METH_FASTCALL, nullptr},
    {"attention", fast(guarded<attention>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding",
                      "Checks and marshalling of the paged-cache calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
