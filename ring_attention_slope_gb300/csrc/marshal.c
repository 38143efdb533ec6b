/*
 * Argument marshalling of the serving calls for Python: torch tensors become
 * slope_tensor descriptors on the C stack and the library is called with them.
 *
 * The smallest of these calls take 3 us on the GPU.  The same marshalling in
 * Python (attributes, struct packing, ctypes) took 6 to 9 us a call on a Grace core,
 * more than everything else on the host but the launch.  Nothing here knows
 * PyTorch's C++ interface: a tensor is asked for dtype, shape, stride(), data_ptr()
 * and get_device() as any Python code would.  Statuses go back as integers.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <stdlib.h>

#include "slope_kv.h"
#include "slope_serving.h"

/* ---------------------------------------------------------------- bound once */

static PyObject *t_bf16, *t_f32, *t_i32;                                /* torch dtypes */
static PyObject *n_dtype, *n_shape, *n_stride, *n_data_ptr, *n_device, *n_numel; /* names */

static struct {
  slope_status (*qk_norm_rope)(const slope_tensor*, const slope_tensor*, const slope_tensor*, const slope_tensor*, int,
                               float, const slope_rope*, const int32_t*, int64_t, slope_tensor*, slope_tensor*, void*);
  slope_status (*attn_varlen)(const slope_tensor*, const slope_tensor*, const slope_tensor*, const int64_t*, int64_t,
                              int, int64_t, float, slope_tensor*, slope_tensor*, void*);
  slope_status (*kv4_write)(const slope_kv4_cache*, const slope_tensor*, const slope_tensor*, const int32_t*, void*);
  slope_status (*kv4_read)(const slope_kv4_cache*, const int32_t*, slope_tensor*, slope_tensor*, void*);
  slope_status (*kv4_attn)(const slope_tensor*, const slope_kv4_cache*, const int32_t*, int64_t, int64_t,
                           const int32_t*, int32_t, int64_t, float, slope_tensor*, slope_tensor*, void*, size_t, void*);
  size_t (*cache_bytes)(int64_t, int32_t, int32_t, int32_t, int32_t);
  size_t (*attn_workspace_size)(int64_t, int64_t, const slope_kv4_cache*, int32_t);
} lib;

static struct { /* the calls of slope_kv.h */
  slope_status (*write)(const slope_kv_cache*, const slope_tensor*, const slope_tensor*, const int32_t*, slope_tensor*,
                        void*);
  slope_status (*attn)(const slope_tensor*, const slope_kv_cache*, const slope_kv_batch*, int64_t, float, slope_tensor*,
                       slope_tensor*, void*, size_t, void*);
  slope_status (*weights)(const slope_tensor*, const slope_kv_cache*, const slope_kv_batch*, const slope_tensor*, int64_t,
                          float, int, slope_tensor*, void*, size_t, void*);
  slope_status (*evict)(const slope_kv_cache*, slope_tensor*, int64_t, const int32_t*, int64_t, int64_t, const int32_t*,
                        int64_t, int64_t, int64_t, const int32_t*, int64_t, int64_t, int32_t*, int32_t*, void*, size_t,
                        void*);
  size_t (*attn_size)(int64_t, int64_t, const slope_kv_cache*, int32_t);
  size_t (*weights_size)(int64_t, int64_t, const slope_kv_cache*, int32_t);
  size_t (*evict_size)(int64_t, int64_t, int64_t);
} kv;

/* bind(bfloat16, float32, int32, addresses of the seven calls in the order above) */
static PyObject* bind(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *a, *b, *c;
  unsigned long long f[7];
  if (!PyArg_ParseTuple(args, "OOOKKKKKKK", &a, &b, &c, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6])) return NULL;
  Py_INCREF(a), Py_INCREF(b), Py_INCREF(c);
  Py_XSETREF(t_bf16, a);
  Py_XSETREF(t_f32, b);
  Py_XSETREF(t_i32, c);
  *(void**)&lib.qk_norm_rope = (void*)(uintptr_t)f[0];
  *(void**)&lib.attn_varlen = (void*)(uintptr_t)f[1];
  *(void**)&lib.kv4_write = (void*)(uintptr_t)f[2];
  *(void**)&lib.kv4_read = (void*)(uintptr_t)f[3];
  *(void**)&lib.kv4_attn = (void*)(uintptr_t)f[4];
  *(void**)&lib.cache_bytes = (void*)(uintptr_t)f[5];
  *(void**)&lib.attn_workspace_size = (void*)(uintptr_t)f[6];
  Py_RETURN_NONE;
}

/* bind_kv(addresses of the seven calls in the order above); bind comes first */
static PyObject* bind_kv(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long f[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6])) return NULL;
  *(void**)&kv.write = (void*)(uintptr_t)f[0];
  *(void**)&kv.attn = (void*)(uintptr_t)f[1];
  *(void**)&kv.weights = (void*)(uintptr_t)f[2];
  *(void**)&kv.evict = (void*)(uintptr_t)f[3];
  *(void**)&kv.attn_size = (void*)(uintptr_t)f[4];
  *(void**)&kv.weights_size = (void*)(uintptr_t)f[5];
  *(void**)&kv.evict_size = (void*)(uintptr_t)f[6];
  Py_RETURN_NONE;
}

/* ---------------------------------------------------------------- arguments */

static int as_i64(PyObject* o, int64_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = v;
  return 0;
}

/* The integer that the tensor's method returns. */
static int ask(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (r == NULL) return -1;
  const int bad = as_i64(r, out);
  Py_DECREF(r);
  return bad;
}

/* Checks that the tensor is on device dev (an empty one may be anywhere): the launch goes to that device's stream. */
static int check_device(PyObject* t, int64_t dev) {
  int64_t on, n;
  if (ask(t, n_device, &on) < 0) return -1;
  if (on == dev) return 0;
  if (ask(t, n_numel, &n) < 0) return -1;
  if (n == 0) return 0;
  if (on < 0)
    PyErr_SetString(PyExc_TypeError, "libslope operates on CUDA tensors");
  else
    PyErr_Format(PyExc_ValueError, "tensor on cuda:%lld, but the current device is cuda:%lld", (long long)on, (long long)dev);
  return -1;
}

/* dst[at ..] = the tuple's entries; returns their number, at most `room`, or -1. */
static Py_ssize_t entries(PyObject* tuple, int64_t* dst, Py_ssize_t at, Py_ssize_t room) {
  if (!PyTuple_Check(tuple)) {
    PyErr_SetString(PyExc_TypeError, "expected a tensor");
    return -1;
  }
  const Py_ssize_t n = PyTuple_GET_SIZE(tuple);
  if (n > room) {
    PyErr_SetString(PyExc_ValueError, "tensors must be rank 2 or 3");
    return -1;
  }
  for (Py_ssize_t i = 0; i < n; ++i)
    if (as_i64(PyTuple_GET_ITEM(tuple, i), &dst[at + i]) < 0) return -1;
  return n;
}

/* Fills *d for a tensor of rank 2 or 3 (or, where `vector` is set, of rank 1, taken as [1, n]) and points *out
 * at it; None leaves *out NULL.  -1 with an exception set. */
static int describe(PyObject* t, int64_t dev, int vector, slope_tensor* d, slope_tensor** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  if (check_device(t, dev) < 0) return -1;
  PyObject* o = PyObject_GetAttr(t, n_dtype);
  if (o == NULL) return -1;
  if (o == t_bf16) {
    d->dtype = SLOPE_BF16;
  } else if (o == t_f32) {
    d->dtype = SLOPE_F32;
  } else {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %S", o);
    Py_DECREF(o);
    return -1;
  }
  Py_DECREF(o);
  o = PyObject_GetAttr(t, n_shape);
  if (o == NULL) return -1;
  Py_ssize_t n = entries(o, d->shape, 0, 3);
  Py_DECREF(o);
  if (n < 0) return -1;
  o = PyObject_CallMethodNoArgs(t, n_stride);
  if (o == NULL) return -1;
  const Py_ssize_t m = entries(o, d->stride, 0, 3);
  Py_DECREF(o);
  if (m < 0) return -1;
  if (n == 1 && vector) {
    d->shape[1] = d->shape[0];
    d->stride[1] = d->stride[0];
    d->shape[0] = 1;
    d->stride[0] = d->shape[1];
    n = 2;
  }
  if (n < 2 || (m != n && !(vector && m == 1))) {
    PyErr_SetString(PyExc_ValueError, "tensors must be rank 2 or 3");
    return -1;
  }
  if (n == 2) d->shape[2] = d->stride[2] = 0;
  d->ndim = (int32_t)n;
  int64_t ptr;
  if (ask(t, n_data_ptr, &ptr) < 0) return -1;
  d->data = (void*)(uintptr_t)ptr;
  *out = d;
  return 0;
}

/* Address of a device int32 array: one dense row of n elements, or, with n < 0, a table. */
static int index_array(PyObject* t, const char* what, int64_t dev, int64_t n, const int32_t** out) {
  PyObject* o = PyObject_GetAttr(t, n_dtype);
  if (o == NULL) return -1;
  const int right = o == t_i32;
  if (!right) PyErr_Format(PyExc_TypeError, "%s must be int32, got %S", what, o);
  Py_DECREF(o);
  if (!right || check_device(t, dev) < 0) return -1;
  if (n >= 0) {
    int64_t shape[3], stride[3];
    o = PyObject_GetAttr(t, n_shape);
    if (o == NULL) return -1;
    const Py_ssize_t rank = entries(o, shape, 0, 3);
    if (rank < 0) {
      Py_DECREF(o);
      return -1;
    }
    if (rank != 1 || shape[0] != n) {
      PyErr_Format(PyExc_ValueError, "%s must have shape [%lld], got %S", what, (long long)n, o);
      Py_DECREF(o);
      return -1;
    }
    Py_DECREF(o);
    if (n > 1) {
      o = PyObject_CallMethodNoArgs(t, n_stride);
      if (o == NULL) return -1;
      const Py_ssize_t m = entries(o, stride, 0, 3);
      Py_DECREF(o);
      if (m < 0) return -1;
      if (stride[0] != 1) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
        return -1;
      }
    }
  }
  int64_t ptr;
  if (ask(t, n_data_ptr, &ptr) < 0) return -1;
  *out = (const int32_t*)(uintptr_t)ptr;
  return 0;
}

/* The structure packed in a bytes object of its size; None is NULL. */
static int structure(PyObject* o, size_t size, const void** out) {
  *out = NULL;
  if (o == Py_None) return 0;
  if (!PyBytes_Check(o) || (size_t)PyBytes_GET_SIZE(o) != size) {
    PyErr_SetString(PyExc_TypeError, "expected a packed structure");
    return -1;
  }
  *out = PyBytes_AS_STRING(o);
  return 0;
}

static int want(Py_ssize_t have, Py_ssize_t n) {
  if (have == n) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, have);
  return -1;
}

static int as_float(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

/* First dimension of a tensor. */
static int rows_of(PyObject* t, int64_t* out) {
  PyObject* o = PyObject_GetAttr(t, n_shape);
  if (o == NULL) return -1;
  int64_t shape[8];
  const Py_ssize_t n = entries(o, shape, 0, 8);
  Py_DECREF(o);
  if (n < 0) return -1;
  *out = n > 0 ? shape[0] : 0;
  return 0;
}

/* ---------------------------------------------------------------- the calls */

/* A library call's status into st, the call made without the interpreter's lock: a launch waits while the stream's
 * queue is full, perhaps for a host function queued there that wants the lock.  What the call reads is on the C
 * stack or belongs to arguments that the caller holds. */
#define UNLOCKED(st, call) \
  do {                     \
    Py_BEGIN_ALLOW_THREADS \
    st = (call);           \
    Py_END_ALLOW_THREADS   \
  } while (0)

/* (q, k, q_weight, k_weight, norm, eps, rope, positions, pos0, q_out, k_out, stream, dev) */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[6], *q, *k, *qw, *kw, *qo, *ko;
  const int32_t* pos = NULL;
  const void* rope;
  int64_t pos0, stream, dev, rows;
  float eps;
  if (want(n, 13) < 0 || as_i64(a[11], &stream) < 0 || as_i64(a[12], &dev) < 0) return NULL;
  const int norm = PyObject_IsTrue(a[4]);
  if (norm < 0 || as_float(a[5], &eps) < 0 || structure(a[6], sizeof(slope_rope), &rope) < 0 || as_i64(a[8], &pos0) < 0)
    return NULL;
  if (describe(a[0], dev, 0, &d[0], &q) < 0 || describe(a[1], dev, 0, &d[1], &k) < 0 ||
      describe(a[2], dev, 1, &d[2], &qw) < 0 || describe(a[3], dev, 1, &d[3], &kw) < 0 ||
      describe(a[9], dev, 0, &d[4], &qo) < 0 || describe(a[10], dev, 0, &d[5], &ko) < 0)
    return NULL;
  rows = q != NULL ? q->shape[0] : k != NULL ? k->shape[0] : 0;
  if (a[7] != Py_None && index_array(a[7], "positions", dev, rows, &pos) < 0) return NULL;
  slope_status st;
  UNLOCKED(st, lib.qk_norm_rope(q, k, qw, kw, norm, eps, (const slope_rope*)rope, pos, pos0, qo, ko,
                                    (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (q, k, v, cu_seqlens as a list or tuple, causal, window, scale, out, lse, stream, dev) */
static PyObject* attn_varlen(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[5], *q, *k, *v, *out, *lse;
  int64_t window, stream, dev, few[256], *cu = few;
  float scale;
  if (want(n, 11) < 0 || as_i64(a[9], &stream) < 0 || as_i64(a[10], &dev) < 0) return NULL;
  const int causal = PyObject_IsTrue(a[4]);
  if (causal < 0 || as_i64(a[5], &window) < 0 || as_float(a[6], &scale) < 0) return NULL;
  if (describe(a[0], dev, 0, &d[0], &q) < 0 || describe(a[1], dev, 0, &d[1], &k) < 0 ||
      describe(a[2], dev, 0, &d[2], &v) < 0 || describe(a[7], dev, 0, &d[3], &out) < 0 ||
      describe(a[8], dev, 0, &d[4], &lse) < 0)
    return NULL;
  // a tuple of its own: reading an entry may run Python code, which may change the caller's list
  PyObject* seq = PySequence_Tuple(a[3]);
  if (seq == NULL) return NULL;
  const Py_ssize_t m = PyTuple_GET_SIZE(seq);
  PyObject* result = NULL;
  if (m < 1) {
    PyErr_SetString(PyExc_ValueError, "cu_seqlens needs at least one entry");
  } else if (m > 256 && (cu = (int64_t*)malloc((size_t)m * sizeof(int64_t))) == NULL) {
    PyErr_NoMemory();
  } else {
    Py_ssize_t i = 0;
    while (i < m && as_i64(PyTuple_GET_ITEM(seq, i), &cu[i]) == 0) ++i;
    if (i == m) {
      slope_status st;
      UNLOCKED(st, lib.attn_varlen(q, k, v, cu, m - 1, causal, window, scale, out, lse, (void*)(uintptr_t)stream));
      result = PyLong_FromLong(st);
    }
  }
  if (cu != few) free(cu);
  Py_DECREF(seq);
  return result;
}

/* (cache, k, v, slots, stream, dev) */
static PyObject* kv4_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[2], *k, *v;
  const int32_t* slots;
  const void* cache;
  int64_t stream, dev;
  if (want(n, 6) < 0 || as_i64(a[4], &stream) < 0 || as_i64(a[5], &dev) < 0) return NULL;
  if (structure(a[0], sizeof(slope_kv4_cache), &cache) < 0 || describe(a[1], dev, 0, &d[0], &k) < 0 ||
      describe(a[2], dev, 0, &d[1], &v) < 0 || index_array(a[3], "slots", dev, k != NULL ? k->shape[0] : 0, &slots) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, lib.kv4_write((const slope_kv4_cache*)cache, k, v, slots, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (cache, slots, k, v, stream, dev) */
static PyObject* kv4_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[2], *k, *v;
  const int32_t* slots;
  const void* cache;
  int64_t stream, dev;
  if (want(n, 6) < 0 || as_i64(a[4], &stream) < 0 || as_i64(a[5], &dev) < 0) return NULL;
  if (structure(a[0], sizeof(slope_kv4_cache), &cache) < 0 || describe(a[2], dev, 0, &d[0], &k) < 0 ||
      describe(a[3], dev, 0, &d[1], &v) < 0 || index_array(a[1], "slots", dev, k != NULL ? k->shape[0] : 0, &slots) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, lib.kv4_read((const slope_kv4_cache*)cache, slots, k, v, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (q, cache, block_table, kv_lens, q_len, window, scale, out, lse, workspace address, workspace bytes, stream, dev) */
static PyObject* kv4_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[3], *q, *out, *lse;
  const int32_t *table, *lens;
  const void* cache;
  int64_t q_len, window, ws, ws_bytes, stream, dev, rows, shape[3], stride[3];
  float scale;
  if (want(n, 13) < 0 || as_i64(a[11], &stream) < 0 || as_i64(a[12], &dev) < 0) return NULL;
  if (structure(a[1], sizeof(slope_kv4_cache), &cache) < 0 || as_i64(a[4], &q_len) < 0 || as_i64(a[5], &window) < 0 ||
      as_float(a[6], &scale) < 0 || as_i64(a[9], &ws) < 0 || as_i64(a[10], &ws_bytes) < 0 || rows_of(a[0], &rows) < 0)
    return NULL;
  if (q_len < 1 || q_len > INT32_MAX || rows % q_len != 0) {
    PyErr_Format(PyExc_ValueError, "q has %lld rows, not a multiple of q_len = %lld", (long long)rows, (long long)q_len);
    return NULL;
  }
  const int64_t batch = rows / q_len;
  PyObject* o = PyObject_GetAttr(a[2], n_shape);
  if (o == NULL) return NULL;
  Py_ssize_t rank = entries(o, shape, 0, 3);
  if (rank >= 0 && (rank != 2 || shape[0] != batch))
    PyErr_Format(PyExc_ValueError, "block_table must have shape [%lld, pages], got %S", (long long)batch, o);
  Py_DECREF(o);
  if (rank != 2 || shape[0] != batch) return NULL;
  o = PyObject_CallMethodNoArgs(a[2], n_stride);
  if (o == NULL) return NULL;
  rank = entries(o, stride, 0, 3);
  Py_DECREF(o);
  if (rank < 0) return NULL;
  if (shape[1] > 1 && stride[1] != 1) {
    PyErr_SetString(PyExc_ValueError, "block_table rows must be contiguous");
    return NULL;
  }
  if (describe(a[0], dev, 0, &d[0], &q) < 0 || describe(a[7], dev, 0, &d[1], &out) < 0 ||
      describe(a[8], dev, 0, &d[2], &lse) < 0 || index_array(a[2], "block_table", dev, -1, &table) < 0 ||
      index_array(a[3], "kv_lens", dev, batch, &lens) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, lib.kv4_attn(q, (const slope_kv4_cache*)cache, table, batch > 1 ? stride[0] : shape[1], shape[1], lens,
                            (int32_t)q_len, window, scale, out, lse, (void*)(uintptr_t)ws, (size_t)ws_bytes,
                            (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

static int as_i32(PyObject* o, int32_t* out) {
  int64_t v;
  if (as_i64(o, &v) < 0) return -1;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_OverflowError, "size out of range");
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

/* (n_pages, page_size, Hkv, dqk, dv) */
static PyObject* cache_bytes(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t pages;
  int32_t v[4];
  if (want(n, 5) < 0 || as_i64(a[0], &pages) < 0) return NULL;
  for (int i = 0; i < 4; ++i)
    if (as_i32(a[i + 1], &v[i]) < 0) return NULL;
  return PyLong_FromSize_t(lib.cache_bytes(pages, v[0], v[1], v[2], v[3]));
}

/* (B, Hq, cache, q_len) */
static PyObject* attn_workspace_size(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t batch, heads;
  int32_t q_len;
  const void* cache;
  if (want(n, 4) < 0 || as_i64(a[0], &batch) < 0 || as_i64(a[1], &heads) < 0 ||
      structure(a[2], sizeof(slope_kv4_cache), &cache) < 0 || as_i32(a[3], &q_len) < 0)
    return NULL;
  return PyLong_FromSize_t(lib.attn_workspace_size(batch, heads, (const slope_kv4_cache*)cache, q_len));
}

/* ---------------------------------------------------------------- the 16-bit cache */

/* A block table [batch, pages]: its address, pages and the distance of its rows. */
static int block_table(PyObject* t, const char* what, int64_t dev, int64_t batch, const int32_t** out, int64_t* pages,
                       int64_t* stride) {
  int64_t shape[3], strides[3];
  PyObject* o = PyObject_GetAttr(t, n_shape);
  if (o == NULL) return -1;
  Py_ssize_t rank = entries(o, shape, 0, 3);
  if (rank >= 0 && (rank != 2 || shape[0] != batch))
    PyErr_Format(PyExc_ValueError, "%s must have shape [%lld, pages], got %S", what, (long long)batch, o);
  Py_DECREF(o);
  if (rank != 2 || shape[0] != batch) return -1;
  o = PyObject_CallMethodNoArgs(t, n_stride);
  if (o == NULL) return -1;
  rank = entries(o, strides, 0, 3);
  Py_DECREF(o);
  if (rank < 0) return -1;
  if (shape[1] > 1 && strides[1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s rows must be contiguous", what);
    return -1;
  }
  *pages = shape[1];
  *stride = batch > 1 ? strides[0] : shape[1];
  return index_array(t, what, dev, -1, out);
}

/* The batch of (block_table, kv_lens, cu_q or None, q_len). */
static int batch_of(PyObject* const* a, int64_t dev, slope_kv_batch* b) {
  if (rows_of(a[1], &b->B) < 0 || block_table(a[0], "block_table", dev, b->B, &b->block_table, &b->max_pages, &b->table_stride) < 0 ||
      index_array(a[1], "kv_lens", dev, b->B, &b->kv_lens) < 0 || as_i32(a[3], &b->q_len) < 0)
    return -1;
  b->cu_q = NULL;
  if (a[2] != Py_None && index_array(a[2], "cu_q", dev, b->B + 1, &b->cu_q) < 0) return -1;
  return 0;
}

/* (cache, k, v, slots, weights, stream, dev) */
static PyObject* kv_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[3], *k, *v, *w;
  const int32_t* slots;
  const void* cache;
  int64_t stream, dev;
  if (want(n, 7) < 0 || as_i64(a[5], &stream) < 0 || as_i64(a[6], &dev) < 0) return NULL;
  if (structure(a[0], sizeof(slope_kv_cache), &cache) < 0 || describe(a[1], dev, 0, &d[0], &k) < 0 ||
      describe(a[2], dev, 0, &d[1], &v) < 0 || describe(a[4], dev, 0, &d[2], &w) < 0 ||
      index_array(a[3], "slots", dev, k != NULL ? k->shape[0] : 0, &slots) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, kv.write((const slope_kv_cache*)cache, k, v, slots, w, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (q, cache, block_table, kv_lens, cu_q, q_len, window, scale, out, lse, workspace address, workspace bytes, stream, dev) */
static PyObject* kv_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[3], *q, *out, *lse;
  slope_kv_batch batch;
  const void* cache;
  int64_t window, ws, ws_bytes, stream, dev;
  float scale;
  if (want(n, 14) < 0 || as_i64(a[12], &stream) < 0 || as_i64(a[13], &dev) < 0) return NULL;
  if (structure(a[1], sizeof(slope_kv_cache), &cache) < 0 || batch_of(&a[2], dev, &batch) < 0 ||
      as_i64(a[6], &window) < 0 || as_float(a[7], &scale) < 0 || as_i64(a[10], &ws) < 0 || as_i64(a[11], &ws_bytes) < 0)
    return NULL;
  if (describe(a[0], dev, 0, &d[0], &q) < 0 || describe(a[8], dev, 0, &d[1], &out) < 0 ||
      describe(a[9], dev, 0, &d[2], &lse) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, kv.attn(q, (const slope_kv_cache*)cache, &batch, window, scale, out, lse, (void*)(uintptr_t)ws,
                       (size_t)ws_bytes, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (q, cache, block_table, kv_lens, cu_q, q_len, lse, window, scale, accumulate, weights, workspace address, workspace
 * bytes, stream, dev) */
static PyObject* kv_attn_weights(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d[3], *q, *lse, *w;
  slope_kv_batch batch;
  const void* cache;
  int64_t window, ws, ws_bytes, stream, dev;
  float scale;
  if (want(n, 15) < 0 || as_i64(a[13], &stream) < 0 || as_i64(a[14], &dev) < 0) return NULL;
  const int accumulate = PyObject_IsTrue(a[9]);
  if (accumulate < 0 || structure(a[1], sizeof(slope_kv_cache), &cache) < 0 || batch_of(&a[2], dev, &batch) < 0 ||
      as_i64(a[7], &window) < 0 || as_float(a[8], &scale) < 0 || as_i64(a[11], &ws) < 0 || as_i64(a[12], &ws_bytes) < 0)
    return NULL;
  if (describe(a[0], dev, 0, &d[0], &q) < 0 || describe(a[6], dev, 0, &d[1], &lse) < 0 ||
      describe(a[10], dev, 0, &d[2], &w) < 0)
    return NULL;
  slope_status st;
  UNLOCKED(st, kv.weights(q, (const slope_kv_cache*)cache, &batch, lse, window, scale, accumulate, w, (void*)(uintptr_t)ws,
                          (size_t)ws_bytes, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (cache, weights, block_table, kv_lens, keep, first, recent, out_table or None, kept, out_lens, workspace address,
 * workspace bytes, stream, dev) */
static PyObject* kv_evict(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  slope_tensor d, *w;
  const int32_t *table, *lens, *out_table = NULL, *kept, *out_lens;
  const void* cache;
  int64_t batch, pages, stride, out_pages = 0, out_stride = 0, keep, first, recent, ws, ws_bytes, stream, dev;
  if (want(n, 14) < 0 || as_i64(a[12], &stream) < 0 || as_i64(a[13], &dev) < 0) return NULL;
  if (structure(a[0], sizeof(slope_kv_cache), &cache) < 0 || describe(a[1], dev, 0, &d, &w) < 0 ||
      rows_of(a[3], &batch) < 0 || block_table(a[2], "block_table", dev, batch, &table, &pages, &stride) < 0 ||
      index_array(a[3], "kv_lens", dev, batch, &lens) < 0 || as_i64(a[4], &keep) < 0 || as_i64(a[5], &first) < 0 ||
      as_i64(a[6], &recent) < 0 || as_i64(a[10], &ws) < 0 || as_i64(a[11], &ws_bytes) < 0)
    return NULL;
  if (a[7] != Py_None && block_table(a[7], "out_table", dev, batch, &out_table, &out_pages, &out_stride) < 0) return NULL;
  if (index_array(a[8], "kept", dev, -1, &kept) < 0 || index_array(a[9], "out_lens", dev, batch, &out_lens) < 0) return NULL;
  slope_status st;
  UNLOCKED(st, kv.evict((const slope_kv_cache*)cache, w, batch, table, stride, pages, lens, keep, first, recent, out_table,
                        out_stride, out_pages, (int32_t*)kept, (int32_t*)out_lens, (void*)(uintptr_t)ws,
                        (size_t)ws_bytes, (void*)(uintptr_t)stream));
  return PyLong_FromLong(st);
}

/* (T, Hq, cache, q_len, weights): the workspace of kv_attn, or with weights that of kv_attn_weights */
static PyObject* kv_attn_workspace_size(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t rows, heads;
  int32_t q_len;
  const void* cache;
  if (want(n, 5) < 0 || as_i64(a[0], &rows) < 0 || as_i64(a[1], &heads) < 0 ||
      structure(a[2], sizeof(slope_kv_cache), &cache) < 0 || as_i32(a[3], &q_len) < 0)
    return NULL;
  const int weights = PyObject_IsTrue(a[4]);
  if (weights < 0) return NULL;
  return PyLong_FromSize_t((weights ? kv.weights_size : kv.attn_size)(rows, heads, (const slope_kv_cache*)cache, q_len));
}

/* (B, Hkv, keep) */
static PyObject* kv_evict_workspace_size(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t batch, heads, keep;
  if (want(n, 3) < 0 || as_i64(a[0], &batch) < 0 || as_i64(a[1], &heads) < 0 || as_i64(a[2], &keep) < 0) return NULL;
  return PyLong_FromSize_t(kv.evict_size(batch, heads, keep));
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "dtypes and addresses of the library's calls"},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"attn_varlen", (PyCFunction)(void (*)(void))attn_varlen, METH_FASTCALL, NULL},
    {"kv4_write", (PyCFunction)(void (*)(void))kv4_write, METH_FASTCALL, NULL},
    {"kv4_read", (PyCFunction)(void (*)(void))kv4_read, METH_FASTCALL, NULL},
    {"kv4_attn", (PyCFunction)(void (*)(void))kv4_attn, METH_FASTCALL, NULL},
    {"cache_bytes", (PyCFunction)(void (*)(void))cache_bytes, METH_FASTCALL, NULL},
    {"attn_workspace_size", (PyCFunction)(void (*)(void))attn_workspace_size, METH_FASTCALL, NULL},
    {"bind_kv", bind_kv, METH_VARARGS, "addresses of the library's calls on the 16-bit cache"},
    {"kv_write", (PyCFunction)(void (*)(void))kv_write, METH_FASTCALL, NULL},
    {"kv_attn", (PyCFunction)(void (*)(void))kv_attn, METH_FASTCALL, NULL},
    {"kv_attn_weights", (PyCFunction)(void (*)(void))kv_attn_weights, METH_FASTCALL, NULL},
    {"kv_evict", (PyCFunction)(void (*)(void))kv_evict, METH_FASTCALL, NULL},
    {"kv_attn_workspace_size", (PyCFunction)(void (*)(void))kv_attn_workspace_size, METH_FASTCALL, NULL},
    {"kv_evict_workspace_size", (PyCFunction)(void (*)(void))kv_evict_workspace_size, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of the serving calls.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  n_dtype = PyUnicode_InternFromString("dtype");
  n_shape = PyUnicode_InternFromString("shape");
  n_stride = PyUnicode_InternFromString("stride");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  n_device = PyUnicode_InternFromString("get_device");
  n_numel = PyUnicode_InternFromString("numel");
  if (!n_dtype || !n_shape || !n_stride || !n_data_ptr || !n_device || !n_numel) return NULL;
  return PyModule_Create(&module);
}
