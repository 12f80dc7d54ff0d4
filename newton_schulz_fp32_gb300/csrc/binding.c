/* Argument marshalling of the embedding and loss calls, in C.
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
