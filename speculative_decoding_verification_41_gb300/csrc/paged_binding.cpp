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

#include "../../include/dspark_q8.h"

namespace {

decltype(&dspark_pages_reserve) g_reserve;
decltype(&dspark_pages_release) g_release;
decltype(&dspark_kv_append) g_append;
decltype(&dspark_paged_attention) g_attention;
decltype(&dspark_rotary) g_rotary;
decltype(&dspark_kv_append_q8) g_append_q8;
decltype(&dspark_kv_gather_q8) g_gather_q8;
decltype(&dspark_paged_attention_q8) g_attention_q8;

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

// ---- the 8-bit cache (include/dspark_q8.h, paged_q8.py)
// [n, heads, D] of a 16-bit type with contiguous rows
bool rows(const at::Tensor* t, int dev, int32_t& dtype) {
  return t && t->is_cuda() && t->get_device() == dev && t->dim() == 3 && t->stride(2) == 1 &&
         t->size(0) <= INT32_MAX && t->size(1) <= INT32_MAX && t->size(2) <= INT32_MAX &&
         element(t->scalar_type(), dtype);
}
bool same(const at::Tensor* a, const at::Tensor* b) {
  return b && a->sizes() == b->sizes() && a->strides() == b->strides() &&
         a->scalar_type() == b->scalar_type() && b->is_cuda() &&
         a->get_device() == b->get_device();
}
struct CacheQ8 {
  int64_t heads, D, page, token, head, spage, sblock, shead;
  int32_t pages, page_size, block;
};
bool cache_q8(const at::Tensor* k, const at::Tensor* v, const at::Tensor* ks, const at::Tensor* vs,
              int dev, CacheQ8& c) {
  if (!k || !ks || k->scalar_type() != at::kFloat8_e4m3fn || k->dim() != 4 || k->stride(3) != 1 ||
      !k->is_cuda() || k->get_device() != dev || !same(k, v) ||
      ks->scalar_type() != at::kFloat || ks->dim() != 3 || !ks->is_cuda() ||
      ks->get_device() != dev || !same(ks, vs))
    return false;
  const int64_t blocks = ks->size(1);
  if (k->size(0) > INT32_MAX || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX ||
      ks->size(0) != k->size(0) || ks->size(2) != k->size(2) || blocks < 1 ||
      k->size(1) % blocks != 0)
    return false;
  c.pages = static_cast<int32_t>(k->size(0)), c.page_size = static_cast<int32_t>(k->size(1));
  c.block = static_cast<int32_t>(k->size(1) / blocks);
  c.heads = k->size(2), c.D = k->size(3);
  c.page = k->stride(0), c.token = k->stride(1), c.head = k->stride(2);
  c.spage = ks->stride(0), c.sblock = ks->stride(1), c.shead = ks->stride(2);
  return true;
}
// positions or slots of n rows at least
bool per_row(const at::Tensor* t, int dev, int64_t n) {
  return plain(t, at::kInt, dev) && t->numel() >= n;
}

// rotary(x, positions, turns, rotation, inverse, out, stream)
PyObject* rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 7 && g_rotary);
  const at::Tensor *x = tensor(a[0]), *pos = tensor(a[1]), *turns = tensor(a[2]), *out = tensor(a[5]);
  REFUSE_UNLESS(x && x->is_cuda());
  const int dev = x->get_device();
  int32_t dtype, odtype;
  int64_t rotation;
  CUstream_st* s;
  const int inverse = PyObject_IsTrue(a[4]);
  if (inverse < 0) return nullptr;
  REFUSE_UNLESS(rows(x, dev, dtype) && rows(out, dev, odtype) && dtype == odtype &&
                x->sizes() == out->sizes() && per_row(pos, dev, x->size(0)) && turns &&
                turns->is_cuda() && turns->get_device() == dev && whole(a[3], rotation) &&
                here(dev) && stream_of(a[6], dev, s));
  return done(g_rotary(x->data_ptr(), x->stride(0), x->stride(1), data<int32_t>(pos),
                       reinterpret_cast<const dspark_rotation*>(rotation), inverse,
                       static_cast<int32_t>(x->size(0)), static_cast<int32_t>(x->size(1)),
                       static_cast<int32_t>(x->size(2)), dtype, out->data_ptr(), out->stride(0),
                       out->stride(1), s));
}

// append_q8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, turns or None, rotation,
//           positions or None, status, stream)
PyObject* append_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 12 && g_append_q8);
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slots = tensor(a[2]),
                   *kc = tensor(a[3]), *status = tensor(a[10]);
  REFUSE_UNLESS(k && kc && kc->is_cuda());
  const int dev = kc->get_device();
  const bool turned = a[7] != Py_None;
  const at::Tensor *turns = turned ? tensor(a[7]) : nullptr, *pos = turned ? tensor(a[9]) : nullptr;
  CacheQ8 c;
  int32_t dtype;
  int64_t rotation = 0;
  CUstream_st* s;
  REFUSE_UNLESS(cache_q8(kc, tensor(a[4]), tensor(a[5]), tensor(a[6]), dev, c));
  REFUSE_UNLESS(rows(k, dev, dtype) && same(k, v) && k->size(1) == c.heads && k->size(2) == c.D &&
                per_row(slots, dev, k->size(0)) && plain(status, at::kInt, dev, 1) &&
                (!turned || (turns && turns->is_cuda() && turns->get_device() == dev &&
                             per_row(pos, dev, k->size(0)) && whole(a[8], rotation))) &&
                here(dev) && stream_of(a[11], dev, s));
  const at::Tensor *vc = tensor(a[4]), *ks = tensor(a[5]), *vs = tensor(a[6]);
  return done(g_append_q8(
      k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1),
      reinterpret_cast<const dspark_rotation*>(rotation), turned ? data<int32_t>(pos) : nullptr,
      data<int32_t>(slots), static_cast<int32_t>(k->size(0)), static_cast<int32_t>(c.heads),
      static_cast<int32_t>(c.D), dtype, kc->data_ptr(), vc->data_ptr(), c.page, c.token, c.head,
      data<float>(ks), data<float>(vs), c.spage, c.sblock, c.shead, c.block, c.page_size, c.pages,
      data<int32_t>(status), s));
}

// gather_q8(k_cache, v_cache, k_scale, v_scale, slot_map, k, v, status, stream)
PyObject* gather_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 9 && g_gather_q8);
  const at::Tensor* t[8];
  for (int i = 0; i < 8; ++i) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[5] && t[0]->is_cuda());
  const int dev = t[0]->get_device();
  CacheQ8 c;
  int32_t dtype;
  CUstream_st* s;
  REFUSE_UNLESS(cache_q8(t[0], t[1], t[2], t[3], dev, c));
  REFUSE_UNLESS(rows(t[5], dev, dtype) && same(t[5], t[6]) && t[5]->size(1) == c.heads &&
                t[5]->size(2) == c.D && per_row(t[4], dev, t[5]->size(0)) &&
                plain(t[7], at::kInt, dev, 1) && here(dev) && stream_of(a[8], dev, s));
  return done(g_gather_q8(t[0]->data_ptr(), t[1]->data_ptr(), c.page, c.token, c.head,
                          data<float>(t[2]), data<float>(t[3]), c.spage, c.sblock, c.shead, c.block,
                          c.page_size, c.pages, data<int32_t>(t[4]),
                          static_cast<int32_t>(t[5]->size(0)), static_cast<int32_t>(c.heads),
                          static_cast<int32_t>(c.D), dtype, t[5]->data_ptr(), t[6]->data_ptr(),
                          t[5]->stride(0), t[5]->stride(1), data<int32_t>(t[7]), s));
}

// attention_q8(q, k_cache, v_cache, k_scale, v_scale, block_table, context_len, row_off, scale,
//              max_new, window, out, lse or None, status, workspace, stream)
PyObject* attention_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  REFUSE_UNLESS(n == 16 && g_attention_q8);
  const at::Tensor* t[15] = {};
  for (int i : {0, 1, 2, 3, 4, 5, 6, 7, 11, 12, 13, 14}) t[i] = tensor(a[i]);
  REFUSE_UNLESS(t[0] && t[1] && t[6] && t[11] && t[14] && t[1]->is_cuda());
  const int dev = t[1]->get_device();
  CacheQ8 c;
  CUstream_st* s;
  REFUSE_UNLESS(cache_q8(t[1], t[2], t[3], t[4], dev, c));
  const at::Tensor& q = *t[0];
  const int64_t B = t[6]->numel();
  int64_t stride;
  int32_t width, max_new, window, dtype;
  const double scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  REFUSE_UNLESS(small(a[9], max_new) && small(a[10], window) && max_new >= 1);
  REFUSE_UNLESS(rows(t[0], dev, dtype) && q.size(2) == c.D && c.heads >= 1 && q.size(1) >= 1 &&
                q.size(1) % c.heads == 0);
  REFUSE_UNLESS(B <= INT32_MAX && plain(t[6], at::kInt, dev, B) &&
                plain(t[7], at::kLong, dev, B + 1) && table(t[5], dev, B, stride, width) &&
                plain(t[11], q.scalar_type(), dev, q.sizes()) &&
                (a[12] == Py_None || plain(t[12], at::kFloat, dev, {q.size(0), q.size(1)})) &&
                plain(t[13], at::kInt, dev, 1) && plain(t[14], at::kByte, dev) && here(dev) &&
                stream_of(a[15], dev, s));
  return done(g_attention_q8(
      q.data_ptr(), q.stride(0), q.stride(1), t[1]->data_ptr(), t[2]->data_ptr(), c.page, c.token,
      c.head, data<float>(t[3]), data<float>(t[4]), c.spage, c.sblock, c.shead, c.block,
      c.page_size, c.pages, data<int32_t>(t[5]), stride, width, data<int32_t>(t[6]),
      data<int64_t>(t[7]), static_cast<int32_t>(B), static_cast<int32_t>(q.size(0)),
      static_cast<int32_t>(q.size(1)), static_cast<int32_t>(c.heads), static_cast<int32_t>(c.D),
      max_new, static_cast<float>(scale), window, dtype, t[11]->data_ptr(),
      a[12] == Py_None ? nullptr : data<float>(t[12]), data<int32_t>(t[13]), t[14]->data_ptr(),
      static_cast<size_t>(t[14]->numel()), s));
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

// bind(reserve, release, append, attention, rotary, append_q8, gather_q8, attention_q8):
// addresses of libdspark's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  int64_t f[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i)
    if (!whole(a[i], f[i])) {
      PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
      return nullptr;
    }
  g_reserve = reinterpret_cast<decltype(g_reserve)>(f[0]);
  g_release = reinterpret_cast<decltype(g_release)>(f[1]);
  g_append = reinterpret_cast<decltype(g_append)>(f[2]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[3]);
  g_rotary = reinterpret_cast<decltype(g_rotary)>(f[4]);
  g_append_q8 = reinterpret_cast<decltype(g_append_q8)>(f[5]);
  g_gather_q8 = reinterpret_cast<decltype(g_gather_q8)>(f[6]);
  g_attention_q8 = reinterpret_cast<decltype(g_attention_q8)>(f[7]);
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
    {"rotary", fast(guarded<rotary>), METH_FASTCALL, nullptr},
    {"append_q8", fast(guarded<append_q8>), METH_FASTCALL, nullptr},
    {"gather_q8", fast(guarded<gather_q8>), METH_FASTCALL, nullptr},
    {"attention_q8", fast(guarded<attention_q8>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_binding",
                      "Checks and marshalling of the paged-cache calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&module); }
