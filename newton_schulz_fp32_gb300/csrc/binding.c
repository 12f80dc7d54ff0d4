/* Argument marshalling of the embedding, loss and layer calls, in C.
 *
 * A call on a few tokens is a few microseconds of GPU time; looking at a dozen
 * tensors' types, shapes and addresses in Python took two to five times that.
 * Each function here takes torch tensors (by their Python interface, so
 * nothing is compiled against torch), checks them, makes the outputs with
 * torch.empty and calls the library on torch's current stream.  A function
 * returns None where the tensors are not on torch's current device: the caller
 * then makes that device current and calls again. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "../../include/muon.h"

/* ------------------------------------------------------------------ state */

static struct {
  PyObject *empty, *raw_stream, *current_device, *error;
  PyObject *bf16, *fp32, *int32, *int64, *uint8;
  PyObject *kw_dtype_device;
  PyObject *s_shape, *s_stride, *s_dtype, *s_device, *s_data_ptr, *s_numel, *s_contiguous, *s_get_device,
      *s_element_size;
  const char* (*last_error)(void);
  int (*embedding)(const void*, int, int64_t, int, int, const void*, int, int64_t, float, void*, int, int64_t, void*);
  int (*embedding_grad_workspace)(int64_t, int, size_t*);
  int (*embedding_grad)(float*, int64_t, const void*, int, int64_t, const void*, int, int64_t, float, int,
                        const muon_param_t*, const muon_partition_t*, int, void*, size_t, void*);
  int (*token_logprobs)(const void*, int, int64_t, int64_t, int, const void*, int, float, float*, void*);
  int (*policy_loss)(const void*, int, int64_t, int64_t, int, const void*, int, const float*, const float*,
                     const float*, const float*, float, float, float, float, float*, float*, void*, int64_t, void*);
  int (*preference_loss_workspace)(int64_t, size_t*);
  int (*preference_loss)(const void*, int, int64_t, int64_t, int, const void*, int, const void*, int, int,
                         const float*, const float*, float, float, float, float*, float*, float*, void*, int64_t,
                         void*, size_t, void*);
  int (*linear_workspace)(const muon_linear_args_t*, size_t*);
  int (*linear)(const muon_linear_args_t*, void*, size_t, void*);
  int (*linear_grad_workspace)(const muon_linear_grad_args_t*, size_t*);
  int (*linear_grad)(const muon_linear_grad_args_t*, void*, size_t, void*);
  int (*dropout)(const void*, int64_t, const void*, int64_t, void*, int64_t, int, int64_t, int, float,
                 const int64_t*, uint32_t, void*);
  int (*norm_rotary)(const muon_heads_t*, int, int, int64_t, int, int, float, const void*, int, int, const double*,
                     const int32_t*, int, int, void*);
  int (*norm_rotary_grad_workspace)(int64_t, int, size_t*);
  int (*norm_rotary_grad)(const muon_heads_grad_t*, int, int, int64_t, int, int, float, const void*, int, int,
                          const double*, const int32_t*, int, int, float*, int64_t, const muon_partition_t*, int,
                          float, int, void*, size_t, void*);
} g;

/* ------------------------------------------------------------------ tensors */

static int refuse(const char* format, const char* name) {
  PyErr_Format(PyExc_ValueError, format, name);
  return -1;
}

/* A method without arguments that returns an integer. */
static int ask(PyObject* t, PyObject* method, long long* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, method);
  if (!r) return -1;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int address(PyObject* t, void** out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, g.s_data_ptr);
  if (!r) return -1;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

static int contiguous(PyObject* t, const char* name) {
  PyObject* r = PyObject_CallMethodNoArgs(t, g.s_contiguous);
  if (!r) return -1;
  const int yes = r == Py_True;
  Py_DECREF(r);
  return yes ? 0 : refuse("%s must be contiguous", name);
}

/* 0 or 1 for the two types a tensor may have. */
static int kind_of(PyObject* t, PyObject* zero, PyObject* one, const char* format, const char* name, int* out) {
  PyObject* d = PyObject_GetAttr(t, g.s_dtype);
  if (!d) return -1;
  const int known = d == zero || d == one;
  *out = d == one;
  Py_DECREF(d);
  return known ? 0 : refuse(format, name);
}

static int element_kind(PyObject* t, const char* name, int* out) {
  return kind_of(t, g.bf16, g.fp32, "%s must be bfloat16 or float32", name, out);
}

static int index_kind(PyObject* t, const char* name, int* out) {
  if (kind_of(t, g.int32, g.int64, "%s must be int32 or int64", name, out)) return -1;
  return contiguous(t, name);
}

typedef struct {
  long long rows, cols, stride;
} Shape;

/* A 2-D tensor whose rows are contiguous. */
static int rows_of(PyObject* t, const char* name, Shape* out) {
  PyObject* shape = PyObject_GetAttr(t, g.s_shape);
  if (!shape) return -1;
  if (!PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != 2) {
    Py_DECREF(shape);
    return refuse("%s must be 2-D", name);
  }
  out->rows = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
  out->cols = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
  Py_DECREF(shape);
  PyObject* stride = PyObject_CallMethodNoArgs(t, g.s_stride);
  if (!stride) return -1;
  if (!PyTuple_Check(stride) || PyTuple_GET_SIZE(stride) != 2) {
    Py_DECREF(stride);
    return refuse("%s must be 2-D", name);
  }
  const long long across = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
  const long long along = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1));
  Py_DECREF(stride);
  if (PyErr_Occurred()) return -1;
  if (along != 1 && out->cols > 1) return refuse("%s's rows must be contiguous", name);
  out->stride = out->rows > 1 || across > out->cols ? across : out->cols;
  return out->rows <= INT64_MAX && out->cols <= INT_MAX ? 0 : refuse("%s has too many columns", name);
}

/* A contiguous float32 tensor of n elements; None gives NULL where `optional`. */
static int per_token(PyObject* t, long long n, int optional, const char* name, void** out) {
  *out = NULL;
  if (t == Py_None && optional) return 0;
  PyObject* d = PyObject_GetAttr(t, g.s_dtype);
  if (!d) return -1;
  const int fp32 = d == g.fp32;
  Py_DECREF(d);
  long long have;
  if (ask(t, g.s_numel, &have)) return -1;
  if (!fp32 || have != n) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous float32 tensor of %lld elements", name, n);
    return -1;
  }
  return contiguous(t, name) ? -1 : address(t, out);
}

/* Where a caller's scratch lies and how many bytes it has. */
static int scratch(PyObject* t, void** out, long long* bytes) {
  long long n, size;
  if (contiguous(t, "workspace") || ask(t, g.s_numel, &n) || ask(t, g.s_element_size, &size) || address(t, out))
    return -1;
  *bytes = n * size;
  return 0;
}

/* 1: all on torch's current device, 0: all on another one, -1: an error.  *device: that device. */
static int placed(PyObject* const* tensors, int n, long long* device) {
  if (ask(tensors[0], g.s_get_device, device)) return -1;
  if (*device < 0) {
    PyErr_SetString(PyExc_ValueError, "tensors must be on a CUDA device");
    return -1;
  }
  for (int i = 1; i < n; ++i) {
    long long d;
    if (!tensors[i] || tensors[i] == Py_None) continue;
    if (ask(tensors[i], g.s_get_device, &d)) return -1;
    if (d != *device) {
      PyErr_SetString(PyExc_ValueError, "every tensor must be on one device");
      return -1;
    }
  }
  PyObject* r = PyObject_CallNoArgs(g.current_device);
  if (!r) return -1;
  const long long now = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (now == -1 && PyErr_Occurred()) return -1;
  return now == *device;
}

static int stream_of(long long device, void** out) {
  PyObject* d = PyLong_FromLongLong(device);
  if (!d) return -1;
  PyObject* r = PyObject_CallOneArg(g.raw_stream, d);
  Py_DECREF(d);
  if (!r) return -1;
  *out = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* torch.empty(size, dtype=dtype, device=like.device); steals `size`. */
static PyObject* make(PyObject* size, PyObject* dtype, PyObject* like) {
  if (!size) return NULL;
  PyObject* device = PyObject_GetAttr(like, g.s_device);
  PyObject* r = NULL;
  if (device) {
    PyObject* args[3] = {size, dtype, device};
    r = PyObject_Vectorcall(g.empty, args, 1, g.kw_dtype_device);
    Py_DECREF(device);
  }
  Py_DECREF(size);
  return r;
}

static PyObject* make_flat(long long n, PyObject* dtype, PyObject* like) {
  return make(PyLong_FromLongLong(n), dtype, like);
}

static PyObject* make_like(PyObject* shaped, PyObject* dtype, PyObject* like) {
  return make(PyObject_GetAttr(shaped, g.s_shape), dtype, like);
}

static int done(int rc) {
  if (rc == 0) return 0;
  PyObject* e = PyObject_CallFunction(g.error, "is", rc, g.last_error());
  if (e) {
    PyErr_SetObject(g.error, e);
    Py_DECREF(e);
  }
  return -1;
}

static int real(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  *out = (float)v;
  return v == -1.0 && PyErr_Occurred() ? -1 : 0;
}

static int arity(Py_ssize_t have, Py_ssize_t want) {
  if (have == want) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, have);
  return -1;
}

/* ------------------------------------------------------------------ calls */

/* embedding(table, ids, scale, out, out_dtype) */
static PyObject* py_embedding(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 5)) return NULL;
  PyObject *table = a[0], *ids = a[1], *out = a[3] == Py_None ? NULL : a[3];
  Shape t, o;
  int tk, ik, ok;
  long long n, have, device;
  float scale;
  void *pt, *pi, *po, *stream;
  if (rows_of(table, "table", &t) || element_kind(table, "table", &tk) || index_kind(ids, "ids", &ik) ||
      ask(ids, g.s_numel, &n) || real(a[2], &scale))
    return NULL;
  if (t.rows > INT_MAX) return refuse("%s has too many rows", "table"), NULL;
  PyObject* tensors[3] = {table, ids, out};
  const int here = placed(tensors, 3, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (out) {
    if (ask(out, g.s_numel, &have)) return NULL;
    PyObject* shape = PyObject_GetAttr(out, g.s_shape);
    if (!shape) return NULL;
    const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
    const long long last = dims ? PyLong_AsLongLong(PyTuple_GET_ITEM(shape, dims - 1)) : -1;
    Py_DECREF(shape);
    PyObject* dtype = PyObject_GetAttr(out, g.s_dtype);
    if (!dtype) return NULL;
    const int other = a[4] != Py_None && a[4] != dtype;
    Py_DECREF(dtype);
    if (last != t.cols || have != n * t.cols || other) {
      PyErr_SetString(PyExc_ValueError, "out must hold ids' shape plus the table's columns");
      return NULL;
    }
    if (dims == 2) {
      if (rows_of(out, "out", &o)) return NULL;
    } else {
      if (contiguous(out, "out (not 2-D)")) return NULL;
      o.stride = t.cols;
    }
    Py_INCREF(out);
  } else {
    PyObject* shape = PyObject_GetAttr(ids, g.s_shape);
    if (!shape) return NULL;
    const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
    PyObject* size = PyTuple_New(dims + 1);
    if (size) {
      for (Py_ssize_t i = 0; i < dims; ++i) {
        PyObject* d = PyTuple_GET_ITEM(shape, i);
        Py_INCREF(d);
        PyTuple_SET_ITEM(size, i, d);
      }
      PyObject* cols = PyLong_FromLongLong(t.cols);
      if (cols) PyTuple_SET_ITEM(size, dims, cols);
      else Py_CLEAR(size);
    }
    Py_DECREF(shape);
    out = make(size, a[4] != Py_None ? a[4] : tk ? g.fp32 : g.bf16, table);
    if (!out) return NULL;
    o.stride = t.cols;
  }
  if (element_kind(out, "out", &ok) || address(table, &pt) || address(ids, &pi) || address(out, &po) ||
      stream_of(device, &stream))
    goto fail;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.embedding(pt, tk, t.stride, (int)t.rows, (int)t.cols, pi, ik, n, scale, po, ok, o.stride, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto fail;
  return out;
fail:
  Py_DECREF(out);
  return NULL;
}

/* embedding_grad(accum, dout, ids, offset, rows, cols, partition table as bytes or None, scale, overwrite,
 *                workspace) */
static PyObject* py_embedding_grad(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 10)) return NULL;
  PyObject *accum = a[0], *dout = a[1], *ids = a[2], *work = a[9] == Py_None ? NULL : a[9];
  Shape d;
  int dk, ik;
  long long n, elems, device, bytes = 0;
  float scale;
  void *pa, *pd, *pi, *pw = NULL, *stream;
  muon_param_t param = {0, 0, 0, 0, 0};
  param.offset = PyLong_AsLongLong(a[3]);
  const long long rows = PyLong_AsLongLong(a[4]), cols = PyLong_AsLongLong(a[5]);
  const int overwrite = PyObject_IsTrue(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (ask(accum, g.s_numel, &elems) || per_token(accum, elems, 0, "accum", &pa) || index_kind(ids, "ids", &ik) ||
      ask(ids, g.s_numel, &n) || rows_of(dout, "dout", &d) || element_kind(dout, "dout", &dk) || real(a[7], &scale))
    return NULL;
  if (d.rows != n || d.cols != cols) return refuse("%s must be tokens x cols", "dout"), NULL;
  if (rows > INT_MAX || rows < INT_MIN) return refuse("%s has too many rows", "the parameter"), NULL;
  param.rows = (int32_t)rows;
  param.cols = (int32_t)cols;
  char* table = NULL;
  Py_ssize_t table_bytes = 0;
  if (a[6] != Py_None && PyBytes_AsStringAndSize(a[6], &table, &table_bytes)) return NULL;
  if (!table && param.offset >= 0 && rows >= 0 && elems - rows * cols < param.offset) {
    PyErr_Format(PyExc_ValueError, "accum holds %lld elements, the parameter begins at %lld and has %lld", elems,
                 (long long)param.offset, rows * cols);
    return NULL;
  }
  PyObject* tensors[4] = {accum, dout, ids, work};
  const int here = placed(tensors, 4, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  size_t need;
  if (done(g.embedding_grad_workspace(n, (int)cols, &need))) return NULL;
  if (work) {
    if (scratch(work, &pw, &bytes)) return NULL;
    Py_INCREF(work);
  } else if (need > 0) {
    work = make_flat((long long)need, g.uint8, accum);
    if (!work) return NULL;
    bytes = (long long)need;
    if (address(work, &pw)) goto fail;
  }
  if (address(dout, &pd) || address(ids, &pi) || stream_of(device, &stream)) goto fail;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.embedding_grad(pa, elems, pd, dk, d.stride, pi, ik, n, scale, overwrite, &param,
                        (const muon_partition_t*)table, (int)(table_bytes / (Py_ssize_t)sizeof(muon_partition_t)), pw,
                        (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto fail;
  Py_XDECREF(work);
  Py_INCREF(accum);
  return accum;
fail:
  Py_XDECREF(work);
  return NULL;
}

/* The rows of logits and targets every loss takes. */
typedef struct {
  Shape z;
  int kind, index;
  long long n;
  void *logits, *targets;
} Rows;

static int loss_rows(PyObject* logits, PyObject* targets, Rows* r) {
  if (rows_of(logits, "logits", &r->z) || element_kind(logits, "logits", &r->kind) ||
      index_kind(targets, "targets", &r->index) || ask(targets, g.s_numel, &r->n))
    return -1;
  if (r->z.rows != r->n) {
    PyErr_SetString(PyExc_ValueError, "one target per row of logits");
    return -1;
  }
  return address(logits, &r->logits) || address(targets, &r->targets) ? -1 : 0;
}

/* The gradient's buffer (a new reference or NULL): as given, a new one (True;
 * its rows lie against 16 bytes as the logits' do, without what lies between
 * those), or none (False, None). */
static int gradient(PyObject* asked, PyObject* logits, const Rows* r, PyObject** out, void** p, long long* stride) {
  *out = NULL;
  *p = NULL;
  *stride = 0;
  if (asked == Py_False || asked == Py_None) return 0;
  if (asked == Py_True) {
    const long long cols = r->z.cols, gap = r->z.rows > 1 && r->z.stride > cols ? r->z.stride - cols : 0;
    const long long wide = cols + gap % (r->kind ? 4 : 8);
    PyObject* d = make(Py_BuildValue("(LL)", r->z.rows, wide), r->kind ? g.fp32 : g.bf16, logits);
    if (d && wide != cols) {
      PyObject* part = PyObject_CallMethod(d, "narrow", "iiL", 1, 0, cols);
      Py_DECREF(d);
      d = part;
    }
    if (!d || address(d, p)) {
      Py_XDECREF(d);
      return -1;
    }
    *out = d;
    *stride = wide;
    return 0;
  }
  Shape s;
  int kind;
  if (rows_of(asked, "dlogits", &s) || element_kind(asked, "dlogits", &kind)) return -1;
  if (kind != r->kind || s.rows != r->z.rows || s.cols != r->z.cols) {
    PyErr_SetString(PyExc_ValueError, "dlogits must match the logits' shape and type");
    return -1;
  }
  if (address(asked, p)) return -1;
  Py_INCREF(asked);
  *out = asked;
  *stride = s.stride;
  return 0;
}

/* token_logprobs(logits, targets, logit_scale, out) */
static PyObject* py_token_logprobs(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 4)) return NULL;
  PyObject* out = a[3] == Py_None ? NULL : a[3];
  Rows r;
  long long device;
  float scale;
  void *po, *stream;
  if (loss_rows(a[0], a[1], &r) || real(a[2], &scale)) return NULL;
  PyObject* tensors[3] = {a[0], a[1], out};
  const int here = placed(tensors, 3, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (out) Py_INCREF(out);
  else if (!(out = make_like(a[1], g.fp32, a[0]))) return NULL;
  if (per_token(out, r.n, 0, "out", &po) || stream_of(device, &stream)) goto fail;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.token_logprobs(r.logits, r.kind, r.z.stride, r.n, (int)r.z.cols, r.targets, r.index, scale, po, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto fail;
  return out;
fail:
  Py_DECREF(out);
  return NULL;
}

/* policy_loss(logits, targets, advantages, weights, old_logp, ref_logp, clip_low, clip_high, kl_coef, logit_scale,
 *             dlogits) */
static PyObject* py_policy_loss(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 11)) return NULL;
  Rows r;
  long long device, dstride;
  float low, high, kl, scale;
  void *adv, *w, *old, *ref, *pd, *ps, *pl, *stream;
  PyObject *d = NULL, *stats = NULL, *logp = NULL, *answer = NULL;
  if (loss_rows(a[0], a[1], &r) || per_token(a[2], r.n, 0, "advantages", &adv) ||
      per_token(a[3], r.n, 0, "weights", &w) || per_token(a[4], r.n, 1, "old_logp", &old) ||
      per_token(a[5], r.n, 1, "ref_logp", &ref) || real(a[6], &low) || real(a[7], &high) || real(a[8], &kl) ||
      real(a[9], &scale))
    return NULL;
  PyObject* tensors[7] = {a[0], a[1], a[2], a[3], a[4], a[5], PyBool_Check(a[10]) ? NULL : a[10]};
  const int here = placed(tensors, 7, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (gradient(a[10], a[0], &r, &d, &pd, &dstride)) return NULL;
  if (!(logp = make_like(a[1], g.fp32, a[0])) || !(stats = make_flat(4, g.fp32, a[0])) || address(logp, &pl) ||
      address(stats, &ps) || stream_of(device, &stream))
    goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.policy_loss(r.logits, r.kind, r.z.stride, r.n, (int)r.z.cols, r.targets, r.index, adv, w, old, ref, low, high,
                     kl, scale, ps, pl, pd, dstride, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  answer = Py_BuildValue("{sOsOsO}", "stats", stats, "logp", logp, "dlogits", d ? d : Py_None);
end:
  Py_XDECREF(d);
  Py_XDECREF(stats);
  Py_XDECREF(logp);
  return answer;
}

/* preference_loss(logits, targets, offsets, ref_logp, beta, label_smoothing, pair_weights, logit_scale, dlogits,
 *                 workspace) */
static PyObject* py_preference_loss(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 10)) return NULL;
  Rows r;
  long long device, dstride, places, bytes = 0;
  int ok;
  float beta, smoothing, scale;
  size_t need;
  void *pf, *ref, *pw, *pd, *ps, *pm, *pl, *pk, *stream;
  PyObject *work = a[9] == Py_None ? NULL : a[9], *d = NULL, *stats = NULL, *margins = NULL, *logp = NULL,
           *answer = NULL;
  if (loss_rows(a[0], a[1], &r) || ask(a[2], g.s_numel, &places)) return NULL;
  if (places % 2 != 1) {
    PyErr_SetString(PyExc_ValueError, "offsets must hold 2 * pairs + 1 positions");
    return NULL;
  }
  const long long pairs = places / 2;
  if (index_kind(a[2], "offsets", &ok) || address(a[2], &pf) || per_token(a[3], r.n, 1, "ref_logp", &ref) ||
      real(a[4], &beta) || real(a[5], &smoothing) || per_token(a[6], pairs, 1, "pair_weights", &pw) ||
      real(a[7], &scale))
    return NULL;
  if (pairs > INT_MAX) return refuse("%s holds too many positions", "offsets"), NULL;
  PyObject* tensors[7] = {a[0], a[1], a[2], a[3], a[6], PyBool_Check(a[8]) ? NULL : a[8], work};
  const int here = placed(tensors, 7, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (done(g.preference_loss_workspace(r.n, &need)) || gradient(a[8], a[0], &r, &d, &pd, &dstride)) return NULL;
  if (work) {
    Py_INCREF(work);
    if (scratch(work, &pk, &bytes)) goto end;
  } else {
    if (!(work = make_flat((long long)need, g.uint8, a[0])) || address(work, &pk)) goto end;
    bytes = (long long)need;
  }
  if (!(logp = make_like(a[1], g.fp32, a[0])) || !(stats = make_flat(4, g.fp32, a[0])) ||
      !(margins = make_flat(pairs, g.fp32, a[0])) || address(logp, &pl) || address(stats, &ps) ||
      address(margins, &pm) || stream_of(device, &stream))
    goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.preference_loss(r.logits, r.kind, r.z.stride, r.n, (int)r.z.cols, r.targets, r.index, pf, ok, (int)pairs, ref,
                         pw, beta, smoothing, scale, ps, pm, pl, pd, dstride, pk, (size_t)bytes, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  answer = Py_BuildValue("{sOsOsOsO}", "stats", stats, "margins", margins, "logp", logp, "dlogits", d ? d : Py_None);
end:
  Py_XDECREF(work);
  Py_XDECREF(d);
  Py_XDECREF(stats);
  Py_XDECREF(margins);
  Py_XDECREF(logp);
  return answer;
}

/* ------------------------------------------------------------------ layers */

/* Scratch of `need` bytes: the caller's (checked by the library) or a new one.
 * *work: a new reference, or NULL where none is needed. */
static int provide(PyObject* given, size_t need, PyObject* like, PyObject** work, void** p, size_t* bytes) {
  *work = NULL;
  *p = NULL;
  *bytes = 0;
  if (given != Py_None) {
    long long have;
    if (scratch(given, p, &have)) return -1;
    *bytes = (size_t)have;
    Py_INCREF(given);
    *work = given;
  } else if (need > 0) {
    if (!(*work = make_flat((long long)need, g.uint8, like))) return -1;
    if (address(*work, p)) {
      Py_CLEAR(*work);
      return -1;
    }
    *bytes = need;
  }
  return 0;
}

/* A bfloat16 matrix. */
static int bf16_rows(PyObject* t, const char* name, Shape* s, void** p) {
  int kind;
  if (rows_of(t, name, s) || element_kind(t, name, &kind)) return -1;
  if (kind) return refuse("%s must be bfloat16", name);
  return address(t, p);
}

/* A matrix of the given shape, and of the given kind if that is not -1. */
static int matrix(PyObject* t, const char* name, long long rows, long long cols, int kind, Shape* s, void** p) {
  int k;
  if (rows_of(t, name, s) || element_kind(t, name, &k)) return -1;
  if (s->rows != rows || s->cols != cols || (kind >= 0 && k != kind)) {
    PyErr_Format(PyExc_ValueError, "%s must be %lld x %lld%s", name, rows, cols,
                 kind < 0 ? "" : kind ? ", float32" : ", bfloat16");
    return -1;
  }
  return address(t, p);
}

/* Two int64: seed and step. */
static int generator(PyObject* t, void** p) {
  *p = NULL;
  if (t == Py_None) return 0;
  PyObject* d = PyObject_GetAttr(t, g.s_dtype);
  if (!d) return -1;
  const int fits = d == g.int64;
  Py_DECREF(d);
  long long n;
  if (ask(t, g.s_numel, &n)) return -1;
  if (!fits || n != 2) return refuse("%s must be a contiguous int64 tensor of 2 elements (seed, step)", "rng");
  return contiguous(t, "rng") ? -1 : address(t, p);
}

static int site_of(PyObject* o, uint32_t* out) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *out = (uint32_t)v;
  return v >= 0 && v <= 0xffffffffll ? 0 : refuse("%s must be in [0, 2^32)", "site");
}

/* A tensor's shape with another last dimension, as a new matrix's size. */
static PyObject* make_rows(long long rows, long long cols, PyObject* dtype, PyObject* like) {
  return make(Py_BuildValue("(LL)", rows, cols), dtype, like);
}

/* Whether a matrix's rows start on 16 bytes: the library then reads it where it lies and needs no scratch. */
static int on16(const void* p, long long rows, long long stride) {
  return (uintptr_t)p % 16 == 0 && (rows <= 1 || (stride % 8 == 0 && stride < (1ll << 39)));
}

/* linear(x, weight, bias, activation, residual, rate, rng, site, out, out_dtype, pre, workspace); x, residual, out and
 * pre are matrices.  Returns out, or (out, pre). */
static PyObject* py_linear(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 12)) return NULL;
  muon_linear_args_t l = {0};
  Shape x, w, s;
  void *p, *pw, *stream;
  long long n, device;
  PyObject *out = NULL, *pre = NULL, *work = NULL, *answer = NULL;
  const int keep_pre = PyBool_Check(a[10]) ? a[10] == Py_True : a[10] != Py_None;
  const long act = PyLong_AsLong(a[3]);
  if (act == -1 && PyErr_Occurred()) return NULL;
  if (bf16_rows(a[0], "x", &x, &p)) return NULL;
  l.x = p;
  if (bf16_rows(a[1], "weight", &w, &p)) return NULL;
  l.weight = p;
  if (w.cols != x.cols) return refuse("%s must be out_features x in_features", "weight"), NULL;
  if (w.rows > INT_MAX) return refuse("%s has too many rows", "weight"), NULL;
  int kind = a[9] == Py_None ? 0 : a[9] == g.fp32 ? 1 : a[9] == g.bf16 ? 0 : -1;
  if (kind < 0) return refuse("%s must be bfloat16 or float32", "out_dtype"), NULL;
  if (a[8] != Py_None) {
    int ok;
    if (element_kind(a[8], "out", &ok)) return NULL;
    if (a[9] != Py_None && ok != kind) return refuse("%s is not of out_dtype", "out"), NULL;
    kind = ok;
  } else if (a[9] == Py_None && a[4] != Py_None && element_kind(a[4], "residual", &kind)) {
    return NULL;
  }
  if (a[2] != Py_None) {
    if (element_kind(a[2], "bias", &l.bias_dtype) || ask(a[2], g.s_numel, &n)) return NULL;
    if (n != w.rows) return refuse("%s must have out_features elements", "bias"), NULL;
    if (contiguous(a[2], "bias") || address(a[2], &p)) return NULL;
    l.bias = p;
  }
  if (a[4] != Py_None) {
    if (matrix(a[4], "residual", x.rows, w.rows, kind, &s, &p)) return NULL;
    l.residual = p;
    l.residual_stride = s.stride;
  }
  if (real(a[5], &l.dropout) || generator(a[6], &p) || site_of(a[7], &l.site)) return NULL;
  l.rng = p;
  PyObject* tensors[8] = {a[0], a[1], a[2], a[4], a[6], a[8], PyBool_Check(a[10]) ? NULL : a[10], a[11]};
  const int here = placed(tensors, 8, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (a[8] != Py_None) {
    if (matrix(a[8], "out", x.rows, w.rows, kind, &s, &p)) return NULL;
    Py_INCREF(a[8]);
    out = a[8];
    l.out_stride = s.stride;
  } else {
    if (!(out = make_rows(x.rows, w.rows, kind ? g.fp32 : g.bf16, a[0])) || address(out, &p)) goto end;
    l.out_stride = w.rows;
  }
  l.out = p;
  if (keep_pre) {
    if (!PyBool_Check(a[10])) {
      if (matrix(a[10], "pre", x.rows, w.rows, 0, &s, &p)) goto end;
      Py_INCREF(a[10]);
      pre = a[10];
      l.pre_stride = s.stride;
    } else {
      if (!(pre = make_rows(x.rows, w.rows, g.bf16, a[0])) || address(pre, &p)) goto end;
      l.pre_stride = w.rows;
    }
    l.pre = x.rows ? p : NULL;
  }
  l.struct_size = (int32_t)sizeof(l);
  l.activation = (int32_t)act;
  l.n_tokens = x.rows;
  l.in_features = (int32_t)x.cols;
  l.out_features = (int32_t)w.rows;
  l.x_stride = x.stride;
  l.weight_stride = w.stride;
  l.out_dtype = kind;
  size_t need = 0, bytes;
  if ((!(on16(l.x, x.rows, x.stride) && on16(l.weight, w.rows, w.stride)) && done(g.linear_workspace(&l, &need))) ||
      provide(a[11], need, a[0], &work, &pw, &bytes) ||
      stream_of(device, &stream))
    goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.linear(&l, pw, bytes, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  if (keep_pre) {
    answer = PyTuple_Pack(2, out, pre);
  } else {
    Py_INCREF(out);
    answer = out;
  }
end:
  Py_XDECREF(out);
  Py_XDECREF(pre);
  Py_XDECREF(work);
  return answer;
}

/* A parameter as a tuple (offset, rows, cols), or None. */
static int param_of(PyObject* o, const char* name, muon_param_t* p, const muon_param_t** out) {
  *out = NULL;
  if (o == Py_None) return 0;
  long long offset, rows, cols;
  if (!PyTuple_Check(o) || !PyArg_ParseTuple(o, "LLL", &offset, &rows, &cols)) {
    if (!PyErr_Occurred()) refuse("%s must be (offset, rows, cols)", name);
    return -1;
  }
  if (rows > INT_MAX || rows < INT_MIN || cols > INT_MAX || cols < INT_MIN)
    return refuse("%s has too many rows or columns", name);
  p->offset = offset;
  p->rows = (int32_t)rows;
  p->cols = (int32_t)cols;
  p->num_heads = p->use_muon = 0;
  *out = p;
  return 0;
}

/* accum and the partition table (bytes or None) a gradient is put in. */
typedef struct {
  void* accum;
  long long elems;
  char* table;
  Py_ssize_t bytes;
  float scale;
  int overwrite;
} Sums;

static int sums_of(PyObject* accum, PyObject* parts, PyObject* scale, PyObject* overwrite, int wanted, Sums* s) {
  *s = (Sums){0};
  if (real(scale, &s->scale)) return -1;
  s->overwrite = PyObject_IsTrue(overwrite);
  if (s->overwrite < 0) return -1;
  if (parts != Py_None && PyBytes_AsStringAndSize(parts, &s->table, &s->bytes)) return -1;
  if (accum == Py_None) return wanted ? refuse("%s is needed for the gradient of a parameter", "accum") : 0;
  return ask(accum, g.s_numel, &s->elems) || per_token(accum, s->elems, 0, "accum", &s->accum) ? -1 : 0;
}

/* linear_grad(accum, dout, x, weight, param, bias_param, partition table, scale, overwrite, activation, pre, dx,
 *             workspace); dout, x, pre and dx are matrices.  Returns dx or None, in a tuple (None means another
 *             device here). */
static PyObject* py_linear_grad(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 13)) return NULL;
  muon_linear_grad_args_t l = {0};
  muon_param_t param, bias;
  Shape d, x, s;
  Sums sums;
  void *p, *pw, *stream;
  long long device;
  PyObject *dx = NULL, *work = NULL, *answer = NULL;
  const int want_dx = PyBool_Check(a[11]) ? a[11] == Py_True : a[11] != Py_None;
  const long act = PyLong_AsLong(a[9]);
  if (act == -1 && PyErr_Occurred()) return NULL;
  if (bf16_rows(a[1], "dout", &d, &p)) return NULL;
  l.dout = p;
  if (param_of(a[4], "param", &param, &l.param) || param_of(a[5], "bias_param", &bias, &l.bias)) return NULL;
  long long in = -1;
  if (a[2] != Py_None) {
    if (bf16_rows(a[2], "x", &x, &p)) return NULL;
    if (x.rows != d.rows) return refuse("%s must have dout's tokens", "x"), NULL;
    l.x = p;
    l.x_stride = x.stride;
    in = x.cols;
  } else if (l.param && d.rows) {
    return refuse("%s is needed for the weight's gradient", "x"), NULL;
  }
  if (a[3] != Py_None) {
    if (bf16_rows(a[3], "weight", &s, &p)) return NULL;
    if (s.rows != d.cols || (in >= 0 && s.cols != in))
      return refuse("%s must be out_features x in_features", "weight"), NULL;
    l.weight = p;
    l.weight_stride = s.stride;
    in = s.cols;
  } else if (want_dx) {
    return refuse("%s is needed for dx", "weight"), NULL;
  }
  if (in < 0) in = l.param ? l.param->cols : 1;
  if (sums_of(a[0], a[6], a[7], a[8], l.param || l.bias, &sums)) return NULL;
  if (want_dx && act != MUON_ACT_NONE) {   /* looked at for the slope alone */
    if (a[10] == Py_None) {
      if (d.rows) return refuse("%s is needed for the activation's slope", "pre"), NULL;
    } else {
      if (matrix(a[10], "pre", d.rows, in, 0, &s, &p)) return NULL;
      l.pre = p;
      l.pre_stride = s.stride;
    }
  }
  PyObject* tensors[7] = {a[1], a[0], a[2], a[3], a[10], PyBool_Check(a[11]) ? NULL : a[11], a[12]};
  const int here = placed(tensors, 7, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (want_dx) {
    if (!PyBool_Check(a[11])) {
      if (matrix(a[11], "dx", d.rows, in, 0, &s, &p)) return NULL;
      Py_INCREF(a[11]);
      dx = a[11];
      l.dx_stride = s.stride;
    } else {
      if (!(dx = make_rows(d.rows, in, g.bf16, a[1])) || address(dx, &p)) goto end;
      l.dx_stride = in;
    }
    l.dx = p;
  }
  l.struct_size = (int32_t)sizeof(l);
  l.activation = (int32_t)act;
  l.n_tokens = d.rows;
  l.in_features = (int32_t)in;
  l.out_features = (int32_t)d.cols;
  l.dout_stride = d.stride;
  l.accum = sums.accum;
  l.accum_elems = sums.elems;
  l.parts = (const muon_partition_t*)sums.table;
  l.nparts = (int32_t)(sums.bytes / (Py_ssize_t)sizeof(muon_partition_t));
  l.scale = sums.scale;
  l.overwrite = sums.overwrite;
  size_t need = 0, bytes;
  if ((!(on16(l.dout, d.rows, d.stride) && on16(l.x, d.rows, l.x_stride) &&
         on16(l.weight, d.cols, l.weight_stride)) &&
       done(g.linear_grad_workspace(&l, &need))) ||
      provide(a[12], need, a[1], &work, &pw, &bytes) ||
      stream_of(device, &stream))
    goto end;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.linear_grad(&l, pw, bytes, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  answer = PyTuple_Pack(1, dx ? dx : Py_None);
end:
  Py_XDECREF(dx);
  Py_XDECREF(work);
  return answer;
}

/* dropout(x, rate, rng, site, residual, out); matrices. */
static PyObject* py_dropout(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 6)) return NULL;
  Shape x, r = {0}, o;
  int kind;
  float rate;
  uint32_t site;
  long long device;
  void *px, *pr = NULL, *po, *rng, *stream;
  PyObject* out;
  if (rows_of(a[0], "x", &x) || element_kind(a[0], "x", &kind) || address(a[0], &px) || real(a[1], &rate) ||
      generator(a[2], &rng) || site_of(a[3], &site) ||
      (a[4] != Py_None && matrix(a[4], "residual", x.rows, x.cols, kind, &r, &pr)))
    return NULL;
  PyObject* tensors[4] = {a[0], a[2], a[4], a[5]};
  const int here = placed(tensors, 4, &device);
  if (here < 0) return NULL;
  if (here == 0) Py_RETURN_NONE;
  if (a[5] != Py_None) {
    if (matrix(a[5], "out", x.rows, x.cols, kind, &o, &po)) return NULL;
    Py_INCREF(a[5]);
    out = a[5];
  } else {
    if (!(out = make_rows(x.rows, x.cols, kind ? g.fp32 : g.bf16, a[0]))) return NULL;
    o.stride = x.cols;
    if (address(out, &po)) goto fail;
  }
  if (stream_of(device, &stream)) goto fail;
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = g.dropout(px, x.stride, pr, r.stride, po, o.stride, kind, x.rows, (int)x.cols, rate, rng, site, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto fail;
  return out;
fail:
  Py_DECREF(out);
  return NULL;
}

/* A tensor of heads: tokens x heads x head_dim, elements of a head contiguous. */
typedef struct {
  long long n, heads, dim, stride, head;
} HeadShape;

static int heads_of(PyObject* t, const char* name, HeadShape* out) {
  PyObject* shape = PyObject_GetAttr(t, g.s_shape);
  if (!shape) return -1;
  PyObject* stride = PyObject_CallMethodNoArgs(t, g.s_stride);
  if (!stride) {
    Py_DECREF(shape);
    return -1;
  }
  const int three = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 3 && PyTuple_Check(stride) &&
                    PyTuple_GET_SIZE(stride) == 3;
  long long along = 1;
  if (three) {
    out->n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    out->heads = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1));
    out->dim = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 2));
    out->stride = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0));
    out->head = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1));
    along = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 2));
  }
  Py_DECREF(shape);
  Py_DECREF(stride);
  if (PyErr_Occurred()) return -1;
  if (!three) return refuse("%s must be tokens x heads x head_dim", name);
  if (along != 1 && out->dim > 1) return refuse("%s's heads must be contiguous", name);
  if (out->heads > INT_MAX || out->dim > INT_MAX) return refuse("%s is too large", name);
  /* strides of dimensions with one element say nothing */
  if (out->heads == 1) out->head = out->dim;
  if (out->n == 1) out->stride = (out->heads - 1) * out->head + out->dim;
  return 0;
}

static int same_heads(PyObject* t, const char* name, const HeadShape* want, int kind, HeadShape* s, void** p) {
  int k;
  if (heads_of(t, name, s) || element_kind(t, name, &k)) return -1;
  if (k != kind || s->n != want->n || s->heads != want->heads || s->dim != want->dim)
    return refuse("%s must have the heads' shape and type", name);
  return address(t, p);
}

static int head_weight(PyObject* t, const char* name, long long dim, int kind, const void** out) {
  *out = NULL;
  if (t == Py_None) return 0;
  int k;
  long long n;
  void* p;
  if (element_kind(t, name, &k) || ask(t, g.s_numel, &n)) return -1;
  if (k != kind || n != dim) return refuse("%s must have head_dim elements of the heads' type", name);
  if (contiguous(t, name) || address(t, &p)) return -1;
  *out = p;
  return 0;
}

/* Whether a buffer is one row of elements of this machine's own type `code`, `size` bytes each. */
static int row_of(const Py_buffer* b, char code, Py_ssize_t size) {
  const char* f = b->format;
  return b->ndim == 1 && b->itemsize == size && f && *f != '>' && *f != '!' && f[strlen(f) - 1] == code;
}

/* positions (tensor or None), inv_freq and axis (buffers of float64 and int32, or None). */
typedef struct {
  void* positions;
  int type, axes, pairs, interleaved, norm;
  float eps;
  Py_buffer freq, axis;
} Turns;

static void turns_gone(Turns* t) {
  if (t->freq.obj) PyBuffer_Release(&t->freq);
  if (t->axis.obj) PyBuffer_Release(&t->axis);
}

static int turns_of(PyObject* positions, PyObject* freq, PyObject* axis, PyObject* interleaved, PyObject* norm,
                    PyObject* eps, long long n, Turns* t) {
  *t = (Turns){0};
  t->axes = 1;
  t->interleaved = PyObject_IsTrue(interleaved);
  t->norm = PyObject_IsTrue(norm);
  if (t->interleaved < 0 || t->norm < 0 || real(eps, &t->eps)) return -1;
  if (freq != Py_None) {
    if (PyObject_GetBuffer(freq, &t->freq, PyBUF_ND | PyBUF_FORMAT)) return -1;
    if (!row_of(&t->freq, 'd', 8)) return refuse("%s must be a 1-D float64 array", "inv_freq");
    if (t->freq.len / 8 > INT_MAX) return refuse("%s is too long", "inv_freq");
    t->pairs = (int)(t->freq.len / 8);
    if (axis != Py_None) {
      if (PyObject_GetBuffer(axis, &t->axis, PyBUF_ND | PyBUF_FORMAT)) return -1;
      if (!row_of(&t->axis, 'i', 4) || t->axis.len / 4 != t->pairs)
        return refuse("%s must be a 1-D int32 array of inv_freq's length", "axis");
    }
  }
  if (positions == Py_None) return t->pairs ? refuse("%s are needed for a rotation", "positions") : 0;
  long long count;
  if (index_kind(positions, "positions", &t->type) || ask(positions, g.s_numel, &count) ||
      address(positions, &t->positions))
    return -1;
  PyObject* shape = PyObject_GetAttr(positions, g.s_shape);
  if (!shape) return -1;
  long long axes = 1;
  if (count != n) {
    const Py_ssize_t dims = PyTuple_GET_SIZE(shape);
    axes = dims ? PyLong_AsLongLong(PyTuple_GET_ITEM(shape, dims - 1)) : -1;
  }
  Py_DECREF(shape);
  if (n == 0 && t->axis.buf) {   /* an empty batch's positions do not tell: as many as the pairs name */
    axes = 1;
    for (int i = 0; i < t->pairs; ++i)
      if (((const int32_t*)t->axis.buf)[i] >= axes) axes = ((const int32_t*)t->axis.buf)[i] + 1ll;
  }
  if (axes < 1 || axes > INT_MAX || count != n * axes)
    return refuse("%s must be one per token, or tokens x axes", "positions");
  t->axes = (int)axes;
  return 0;
}

static PyObject* new_heads(const HeadShape* s, int kind, PyObject* like) {
  return make(Py_BuildValue("(LLL)", s->n, s->heads, s->dim), kind ? g.fp32 : g.bf16, like);
}

/* norm_rotary(q, k, positions, inv_freq, axis, interleaved, norm, q_weight, k_weight, eps, q_out, k_out); returns
 * (q, k or None). */
static PyObject* py_norm_rotary(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 12)) return NULL;
  muon_heads_t h[2] = {{0}, {0}};
  HeadShape s[2], o;
  Turns t = {0};
  int kind, rc = 0;
  long long device;
  void *p, *stream;
  PyObject *outs[2] = {NULL, NULL}, *answer = NULL;
  static const char* const names[2][3] = {{"q", "q_weight", "q_out"}, {"k", "k_weight", "k_out"}};
  const int groups = a[1] == Py_None ? 1 : 2;
  if (element_kind(a[0], "q", &kind)) return NULL;
  for (int i = 0; i < groups; ++i) {
    int other;
    if (heads_of(a[i], names[i][0], &s[i]) || element_kind(a[i], names[i][0], &other) || address(a[i], &p)) return NULL;
    if (other != kind || s[i].n != s[0].n || s[i].dim != s[0].dim)
      return refuse("%s must have q's tokens, head_dim and type", names[i][0]), NULL;
    h[i].x = p;
    h[i].x_stride = s[i].stride;
    h[i].x_head_stride = s[i].head;
    h[i].heads = (int32_t)s[i].heads;
    if (head_weight(a[7 + i], names[i][1], s[0].dim, kind, &h[i].weight)) return NULL;
  }
  if (turns_of(a[2], a[3], a[4], a[5], a[6], a[9], s[0].n, &t)) goto end;
  PyObject* tensors[7] = {a[0], a[1], a[2], a[7], a[8], a[10], a[11]};
  const int here = placed(tensors, 7, &device);
  if (here < 0) goto end;
  if (here == 0) {
    turns_gone(&t);
    Py_RETURN_NONE;
  }
  for (int i = 0; i < groups; ++i) {
    if (a[10 + i] != Py_None) {
      if (same_heads(a[10 + i], names[i][2], &s[i], kind, &o, &p)) goto end;
      Py_INCREF(a[10 + i]);
      outs[i] = a[10 + i];
    } else {
      if (!(outs[i] = new_heads(&s[i], kind, a[0])) || address(outs[i], &p)) goto end;
      o.head = s[i].dim;
      o.stride = s[i].heads * s[i].dim;
    }
    h[i].out = p;
    h[i].out_stride = o.stride;
    h[i].out_head_stride = o.head;
  }
  if (stream_of(device, &stream)) goto end;
  Py_BEGIN_ALLOW_THREADS
  rc = g.norm_rotary(h, groups, kind, s[0].n, (int)s[0].dim, t.norm, t.eps, t.positions, t.type, t.axes, t.freq.buf,
                     t.axis.buf, t.pairs, t.interleaved, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  answer = PyTuple_Pack(2, outs[0], outs[1] ? outs[1] : Py_None);
end:
  turns_gone(&t);
  Py_XDECREF(outs[0]);
  Py_XDECREF(outs[1]);
  return answer;
}

/* norm_rotary_grad(dq, q, dk, k, positions, inv_freq, axis, interleaved, norm, q_weight, k_weight, eps, accum, q_param,
 *                  k_param, partition table, scale, overwrite, dq_out, dk_out, workspace); returns (dq, dk or None). */
static PyObject* py_norm_rotary_grad(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 21)) return NULL;
  muon_heads_grad_t h[2] = {{0}, {0}};
  muon_param_t params[2];
  HeadShape s[2], o;
  Turns t = {0};
  Sums sums;
  int kind, rc = 0;
  long long device;
  size_t need = 0, bytes;
  void *p, *pw, *stream;
  PyObject *outs[2] = {NULL, NULL}, *work = NULL, *answer = NULL;
  static const char* const names[2][5] = {{"dq", "q", "q_weight", "q_param", "dq_out"},
                                          {"dk", "k", "k_weight", "k_param", "dk_out"}};
  const int groups = a[2] == Py_None ? 1 : 2;
  if (element_kind(a[0], "dq", &kind)) return NULL;
  for (int i = 0; i < groups; ++i) {
    int other;
    if (heads_of(a[2 * i], names[i][0], &s[i]) || element_kind(a[2 * i], names[i][0], &other) ||
        address(a[2 * i], &p))
      return NULL;
    if (other != kind || s[i].n != s[0].n || s[i].dim != s[0].dim)
      return refuse("%s must have dq's tokens, head_dim and type", names[i][0]), NULL;
    h[i].dout = p;
    h[i].dout_stride = s[i].stride;
    h[i].dout_head_stride = s[i].head;
    h[i].heads = (int32_t)s[i].heads;
    if (a[2 * i + 1] != Py_None) {
      if (same_heads(a[2 * i + 1], names[i][1], &s[i], kind, &o, &p)) return NULL;
      h[i].x = p;
      h[i].x_stride = o.stride;
      h[i].x_head_stride = o.head;
    }
    if (head_weight(a[9 + i], names[i][2], s[0].dim, kind, &h[i].weight) ||
        param_of(a[13 + i], names[i][3], &params[i], &h[i].param))
      return NULL;
  }
  if (sums_of(a[12], a[15], a[16], a[17], h[0].param || h[1].param, &sums)) return NULL;
  if (turns_of(a[4], a[5], a[6], a[7], a[8], a[11], s[0].n, &t)) goto end;
  PyObject* tensors[11] = {a[0], a[1], a[2], a[3], a[4], a[9], a[10], a[12], a[18], a[19], a[20]};
  const int here = placed(tensors, 11, &device);
  if (here < 0) goto end;
  if (here == 0) {
    turns_gone(&t);
    Py_RETURN_NONE;
  }
  for (int i = 0; i < groups; ++i) {
    if (a[18 + i] != Py_None) {
      if (same_heads(a[18 + i], names[i][4], &s[i], kind, &o, &p)) goto end;
      Py_INCREF(a[18 + i]);
      outs[i] = a[18 + i];
    } else {
      if (!(outs[i] = new_heads(&s[i], kind, a[0])) || address(outs[i], &p)) goto end;
      o.head = s[i].dim;
      o.stride = s[i].heads * s[i].dim;
    }
    h[i].dx = p;
    h[i].dx_stride = o.stride;
    h[i].dx_head_stride = o.head;
  }
  if (((h[0].param || h[1].param) && done(g.norm_rotary_grad_workspace(s[0].n, (int)s[0].dim, &need))) ||
      provide(a[20], need, a[0], &work, &pw, &bytes) || stream_of(device, &stream))
    goto end;
  Py_BEGIN_ALLOW_THREADS
  rc = g.norm_rotary_grad(h, groups, kind, s[0].n, (int)s[0].dim, t.norm, t.eps, t.positions, t.type, t.axes,
                          t.freq.buf, t.axis.buf, t.pairs, t.interleaved, sums.accum, sums.elems,
                          (const muon_partition_t*)sums.table,
                          (int)(sums.bytes / (Py_ssize_t)sizeof(muon_partition_t)), sums.scale, sums.overwrite, pw,
                          bytes, stream);
  Py_END_ALLOW_THREADS
  if (done(rc)) goto end;
  answer = PyTuple_Pack(2, outs[0], outs[1] ? outs[1] : Py_None);
end:
  turns_gone(&t);
  Py_XDECREF(outs[0]);
  Py_XDECREF(outs[1]);
  Py_XDECREF(work);
  return answer;
}

/* ------------------------------------------------------------------ set-up */

static int keep(PyObject** slot, PyObject* from, const char* name) {
  PyObject* v = PyObject_GetAttrString(from, name);
  if (!v) return -1;
  Py_XSETREF(*slot, v);
  return 0;
}

static int entry(PyObject* table, const char* name, void** out) {
  PyObject* v = PyDict_GetItemString(table, name);
  if (!v) {
    PyErr_SetString(PyExc_KeyError, name);
    return -1;
  }
  *out = PyLong_AsVoidPtr(v);
  return *out == NULL ? (PyErr_Occurred() ? -1 : refuse("%s has no address", name)) : 0;
}

/* init(torch, current device of torch, its raw stream on a device, error class,
 *      {name: address of the library's function}) */
static PyObject* py_init(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 5)) return NULL;
  if (keep(&g.empty, a[0], "empty") || keep(&g.bf16, a[0], "bfloat16") || keep(&g.fp32, a[0], "float32") ||
      keep(&g.int32, a[0], "int32") || keep(&g.int64, a[0], "int64") || keep(&g.uint8, a[0], "uint8"))
    return NULL;
  Py_INCREF(a[1]);
  Py_XSETREF(g.current_device, a[1]);
  Py_INCREF(a[2]);
  Py_XSETREF(g.raw_stream, a[2]);
  Py_INCREF(a[3]);
  Py_XSETREF(g.error, a[3]);
#define ENTRY(slot, name) entry(a[4], name, (void**)&g.slot)
  if (ENTRY(last_error, "muon_last_error") || ENTRY(embedding, "muon_embedding") ||
      ENTRY(embedding_grad_workspace, "muon_embedding_grad_workspace") ||
      ENTRY(embedding_grad, "muon_embedding_grad") || ENTRY(token_logprobs, "muon_token_logprobs") ||
      ENTRY(policy_loss, "muon_policy_loss") || ENTRY(preference_loss_workspace, "muon_preference_loss_workspace") ||
      ENTRY(preference_loss, "muon_preference_loss"))
    return NULL;
  Py_RETURN_NONE;
}

/* init_layers({name: address of the library's function}), after init */
static PyObject* py_init_layers(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  if (arity(na, 1)) return NULL;
#undef ENTRY
#define ENTRY(slot) entry(a[0], "muon_" #slot, (void**)&g.slot)
  if (ENTRY(linear_workspace) || ENTRY(linear) || ENTRY(linear_grad_workspace) || ENTRY(linear_grad) ||
      ENTRY(dropout) || ENTRY(norm_rotary) || ENTRY(norm_rotary_grad_workspace) || ENTRY(norm_rotary_grad))
    return NULL;
#undef ENTRY
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))py_init, METH_FASTCALL, NULL},
    {"embedding", (PyCFunction)(void (*)(void))py_embedding, METH_FASTCALL, NULL},
    {"embedding_grad", (PyCFunction)(void (*)(void))py_embedding_grad, METH_FASTCALL, NULL},
    {"token_logprobs", (PyCFunction)(void (*)(void))py_token_logprobs, METH_FASTCALL, NULL},
    {"policy_loss", (PyCFunction)(void (*)(void))py_policy_loss, METH_FASTCALL, NULL},
    {"preference_loss", (PyCFunction)(void (*)(void))py_preference_loss, METH_FASTCALL, NULL},
    {"init_layers", (PyCFunction)(void (*)(void))py_init_layers, METH_FASTCALL, NULL},
    {"linear", (PyCFunction)(void (*)(void))py_linear, METH_FASTCALL, NULL},
    {"linear_grad", (PyCFunction)(void (*)(void))py_linear_grad, METH_FASTCALL, NULL},
    {"dropout", (PyCFunction)(void (*)(void))py_dropout, METH_FASTCALL, NULL},
    {"norm_rotary", (PyCFunction)(void (*)(void))py_norm_rotary, METH_FASTCALL, NULL},
    {"norm_rotary_grad", (PyCFunction)(void (*)(void))py_norm_rotary_grad, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
#define NAME(slot, text) \
  if (!(g.slot = PyUnicode_InternFromString(text))) return NULL
  NAME(s_shape, "shape");
  NAME(s_stride, "stride");
  NAME(s_dtype, "dtype");
  NAME(s_device, "device");
  NAME(s_data_ptr, "data_ptr");
  NAME(s_numel, "numel");
  NAME(s_contiguous, "is_contiguous");
  NAME(s_get_device, "get_device");
  NAME(s_element_size, "element_size");
#undef NAME
  g.kw_dtype_device = Py_BuildValue("(ss)", "dtype", "device");
  if (!g.kw_dtype_device) return NULL;
  return PyModule_Create(&module);
}
