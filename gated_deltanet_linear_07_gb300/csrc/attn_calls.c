/*
 * attn_calls.c -- marshalling of the full-attention calls for Python (CPython C
 * API): tensors' shapes, strides, types and addresses go into the structs of
 * include/gdn.h, outputs are allocated, a non-zero gdn_status comes back as
 * GdnError.  The calls are short (a decode step's kernels take microseconds), and
 * through ctypes the marshalling alone took longer than most of them.
 *
 * It knows tensors only by their Python attributes, so it needs no torch headers;
 * setup() hands it torch's types and functions and the library's entry points.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "gdn.h"

static PyObject *s_shape, *s_stride, *s_dtype, *s_data_ptr, *s_numel, *s_is_contiguous, *s_device,
    *s_get_device, *s_element_size, *s_handle;
static PyObject* io_types[3]; /* by gdn_dtype */
static PyObject *t_int32, *t_float64, *f_empty, *f_empty_on, *f_stream, *f_device, *c_error,
    *empty_kw;

typedef int (*norm_rope_fn)(const gdn_attn_dims*, const gdn_rope_params*, const gdn_view*,
                            const gdn_view*, const int32_t*, int64_t, void*, void*, gdn_stream_t);
typedef int (*append_fn)(const gdn_attn_dims*, const gdn_rope_params*, const gdn_view*,
                         const gdn_view*, const gdn_view*, const int32_t*, const int32_t*, int64_t,
                         const gdn_kv_cache*, void*, void*, int32_t*, gdn_stream_t);
typedef int (*prefill_fn)(const gdn_attn_dims*, const gdn_view*, const gdn_view*, const gdn_view*,
                          const int32_t*, const int32_t*, int32_t, int64_t, int64_t,
                          const gdn_view*, void*, int32_t*, gdn_stream_t);
typedef int (*decode_fn)(const gdn_attn_dims*, const gdn_view*, const gdn_kv_cache*, const int32_t*,
                         int32_t, int64_t, const gdn_view*, void*, void*, size_t, int32_t*,
                         gdn_stream_t);
typedef int (*norm_rope_axes_fn)(const gdn_attn_dims*, const gdn_rope_params*, const gdn_rope_axes*,
                                 const gdn_view*, const gdn_view*, const int32_t*, int64_t, void*,
                                 void*, gdn_stream_t);
typedef int (*kv8_append_fn)(const gdn_attn_dims*, const gdn_rope_params*, const gdn_rope_axes*,
                             const gdn_view*, const gdn_view*, const gdn_view*, const int32_t*,
                             const int32_t*, const int32_t*, int32_t, int64_t,
                             const gdn_kv8_cache*, void*, void*, int32_t*, gdn_stream_t);
typedef int (*kv8_gather_fn)(const gdn_attn_dims*, const gdn_kv8_cache*, const int32_t*, int32_t,
                             int64_t, void*, void*, int32_t*, gdn_stream_t);
typedef int (*decode_kv8_fn)(const gdn_attn_dims*, const gdn_view*, const gdn_kv8_cache*,
                             const int32_t*, int32_t, const gdn_view*, float*, void*, void*, size_t,
                             int32_t*, gdn_stream_t);
typedef int (*kv8_evict_fn)(const gdn_attn_dims*, const gdn_kv8_cache*, const float*,
                            const int32_t*, int32_t, int32_t, int32_t, int32_t,
                            const gdn_kv8_cache*, float*, int32_t*, int32_t*, int32_t*,
                            gdn_stream_t);
static norm_rope_fn call_norm_rope;
static append_fn call_append;
static prefill_fn call_prefill;
static decode_fn call_decode;
/* Of the 8-bit cache and its positions (setup_kv8). */
static PyObject* t_e4m3;
static norm_rope_axes_fn call_norm_rope_axes;
static kv8_append_fn call_kv8_append;
static kv8_gather_fn call_kv8_gather;
static decode_kv8_fn call_decode_kv8;
static kv8_evict_fn call_kv8_evict;

/* ---- attributes of a tensor (0: fine; -1: an exception is set) ---------------- */

static int method_int(PyObject* t, PyObject* name, int64_t* out) {
  PyObject* v = PyObject_CallMethodNoArgs(t, name);
  if (!v) return -1;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}
static int address(PyObject* t, void** out) {
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!v) return -1;
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return !*out && PyErr_Occurred() ? -1 : 0;
}
static int check_dtype(PyObject* t, const char* name, PyObject* want) {
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) return -1;
  const int same = v == want;
  if (!same) PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, want, v);
  Py_DECREF(v);
  return same ? 0 : -1;
}
/* The kernels read memory of the current device: a tensor of the host or of another
   device is refused, once everything else about the call's tensors is right.  (Calls
   hold the interpreter lock throughout.) */
static const char *host_tensor, *odd_tensor;
static int64_t call_device, odd_device; /* of the call's first device tensor; < 0: none so far */
static int note_device(PyObject* t, const char* name) {
  int64_t d;
  if (method_int(t, s_get_device, &d)) return -1;
  if (d < 0) {
    if (!host_tensor) host_tensor = name;
  } else if (call_device < 0) {
    call_device = d;
  } else if (d != call_device && !odd_tensor) {
    odd_tensor = name;
    odd_device = d;
  }
  return 0;
}
static int all_device(void) {
  if (host_tensor) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", host_tensor);
    return -1;
  }
  if (odd_tensor) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%lld, tensors before it on cuda:%lld", odd_tensor,
                 (long long)odd_device, (long long)call_device);
    return -1;
  }
  return 0;
}
/* The integers of a tuple, four at most; their number, or -1. */
static int integers(PyObject* seq, int64_t dims[4]) {
  if (!seq) return -1;
  int n = -1;
  if (!PyTuple_Check(seq)) {
    PyErr_SetString(PyExc_TypeError, "a tensor was expected");
  } else {
    const Py_ssize_t size = PyTuple_GET_SIZE(seq);
    n = (int)size;
    for (Py_ssize_t i = 0; i < size && i < 4; ++i) {
      dims[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
      if (dims[i] == -1 && PyErr_Occurred()) n = -1;
    }
  }
  Py_DECREF(seq);
  return n;
}
static int shape_of(PyObject* t, int64_t dims[4]) {
  return integers(PyObject_GetAttr(t, s_shape), dims);
}

/* ---- arguments ------------------------------------------------------------------ */

/* A [n][heads][d] tensor whose channels are contiguous; None: no data. */
static int view(PyObject* t, const char* name, PyObject* dtype, int64_t n, int64_t heads, int64_t d,
                gdn_view* v) {
  memset(v, 0, sizeof(*v));
  if (t == Py_None) return 0;
  int64_t dims[4], strides[4];
  const int nd = shape_of(t, dims);
  if (nd < 0) return -1;
  if (nd != 3 || dims[0] != n || dims[1] != heads || dims[2] != d) {
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    if (shape)
      PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld, %lld], got %R", name, (long long)n,
                   (long long)heads, (long long)d, shape);
    Py_XDECREF(shape);
    return -1;
  }
  if (check_dtype(t, name, dtype)) return -1;
  if (integers(PyObject_CallMethodNoArgs(t, s_stride), strides) < 0) return -1;
  if (strides[2] != 1) {
    PyErr_Format(PyExc_ValueError, "%s's channels must be contiguous", name);
    return -1;
  }
  void* p;
  if (note_device(t, name) || address(t, &p)) return -1;
  v->data = p;
  v->token_stride = strides[0];
  v->head_stride = strides[1];
  return 0;
}

/* Address of a contiguous tensor of this type and size; None: null. */
static int flat(PyObject* t, const char* name, PyObject* dtype, int64_t numel, void** p) {
  *p = NULL;
  if (t == Py_None) return 0;
  if (check_dtype(t, name, dtype)) return -1;
  int64_t n;
  if (method_int(t, s_numel, &n)) return -1;
  if (n != numel) {
    PyErr_Format(PyExc_ValueError, "%s has %lld elements, expected %lld", name, (long long)n,
                 (long long)numel);
    return -1;
  }
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!c) return -1;
  const int contiguous = PyObject_IsTrue(c);
  Py_DECREF(c);
  if (contiguous != 1) {
    if (contiguous == 0) PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return -1;
  }
  return note_device(t, name) || address(t, p) ? -1 : 0;
}

/* An output of this shape (new reference) and its address, allocated beside `like` when
   None: from the current stream's memory, or, where the call goes to another stream,
   from that one's (a block of the current stream's may still be in use there, and may be
   used there again before the call has run). */
static PyObject* shaped(PyObject* t, const char* name, PyObject* dtype, PyObject* size,
                        int64_t numel, PyObject* like, PyObject* other, void** p) {
  if (!size) return NULL;
  if (t != Py_None) {
    if (flat(t, name, dtype, numel, p) || all_device()) return NULL;
    Py_INCREF(t);
    return t;
  }
  PyObject* made = NULL;
  PyObject* device = PyObject_GetAttr(like, s_device);
  if (device) {
    PyObject* args[4] = {size, dtype, device, other};
    made = other == Py_None ? PyObject_Vectorcall(f_empty, args, 1, empty_kw)
                            : PyObject_Vectorcall(f_empty_on, args, 4, NULL);
  }
  Py_XDECREF(device);
  if (made && address(made, p)) Py_CLEAR(made);
  return made;
}
static PyObject* output(PyObject* t, const char* name, PyObject* dtype, int64_t n, int64_t heads,
                        int64_t d, PyObject* like, PyObject* other, void** p) {
  PyObject* size = Py_BuildValue("(LLL)", (long long)n, (long long)heads, (long long)d);
  PyObject* made = shaped(t, name, dtype, size, n * heads * d, like, other, p);
  Py_XDECREF(size);
  return made;
}

static int dims_of(PyObject* o, gdn_attn_dims* d, PyObject** dtype) {
  host_tensor = odd_tensor = NULL;
  call_device = -1;
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) return -1;
  const int fits = b.len == (Py_ssize_t)sizeof(*d);
  if (fits) memcpy(d, b.buf, sizeof(*d));
  PyBuffer_Release(&b);
  if (!fits) {
    PyErr_SetString(PyExc_TypeError, "dims must be a gdn_attn_dims");
    return -1;
  }
  *dtype = io_types[d->io >= 0 && d->io < 3 ? d->io : 0]; /* the library refuses others */
  return 0;
}

/* The stream given, else the current one of the tensors' device, which has to be the
   current device: the launch goes there.  *other: a given stream that is not the
   current one (borrowed), else None. */
static int stream_of(PyObject* stream, gdn_stream_t* s, PyObject** other) {
  *other = Py_None;
  PyObject* v = PyObject_CallNoArgs(f_device);
  if (!v) return -1;
  const long long now = PyLong_AsLongLong(v);
  if (now != call_device) {
    if (!PyErr_Occurred())
      PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%lld, the current device is cuda:%lld",
                   (long long)call_device, now);
    Py_DECREF(v);
    return -1;
  }
  Py_SETREF(v, PyObject_CallOneArg(f_stream, v));
  if (!v) return -1;
  void* current = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  *s = (gdn_stream_t)current;
  if (!current && PyErr_Occurred()) return -1;
  if (stream == Py_None) return 0;
  if (!(v = PyNumber_Long(stream))) return -1;
  *s = (gdn_stream_t)PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!*s && PyErr_Occurred()) return -1;
  if ((void*)*s != current) *other = stream;
  return 0;
}

static int rope_params(PyObject* const* a, const gdn_attn_dims* d, PyObject* scale,
                       gdn_rope_params* p) {
  void *q, *k, *f;
  if (flat(a[0], "q_norm", io_types[GDN_FP32], d->d, &q) ||
      flat(a[1], "k_norm", io_types[GDN_FP32], d->d, &k) ||
      flat(a[2], "inv_freq", t_float64, d->rot_dim / 2, &f))
    return -1;
  p->q_norm = q;
  p->k_norm = k;
  p->inv_freq = f;
  p->rope_scale = (float)PyFloat_AsDouble(scale);
  p->d_status = NULL;
  return PyErr_Occurred() ? -1 : 0;
}

static int cache_of(PyObject* const* a, const gdn_attn_dims* d, PyObject* dtype, gdn_kv_cache* c) {
  int64_t k[4], t[4];
  const int nk = shape_of(a[0], k);
  if (nk < 0) return -1;
  if (nk != 4 || k[1] != d->h_kv || k[2] != d->page_size || k[3] != d->d) {
    PyErr_Format(PyExc_ValueError, "k_cache must be [num_pages, %d, %d, %d]", d->h_kv, d->page_size,
                 d->d);
    return -1;
  }
  const int nt = shape_of(a[2], t);
  if (nt < 0) return -1;
  if (nt != 2 || t[0] > INT32_MAX || t[1] > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "block_table must be [num_seqs, pages_per_seq]");
    return -1;
  }
  const int64_t numel = k[0] * k[1] * k[2] * k[3];
  void* table;
  if (flat(a[0], "k_cache", dtype, numel, &c->k) || flat(a[1], "v_cache", dtype, numel, &c->v) ||
      flat(a[2], "block_table", t_int32, t[0] * t[1], &table))
    return -1;
  c->block_table = table;
  c->num_pages = k[0];
  c->num_seqs = (int32_t)t[0];
  c->pages_per_seq = (int32_t)t[1];
  return 0;
}

/* Address and bytes of a workspace of any type; None: null. */
static int workspace_of(PyObject* t, void** p, size_t* bytes) {
  int64_t size = 0, item = 0;
  *p = NULL;
  *bytes = 0;
  if (t == Py_None) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  const int contiguous = c ? PyObject_IsTrue(c) : -1;
  Py_XDECREF(c);
  if (contiguous == 0) PyErr_SetString(PyExc_ValueError, "workspace must be contiguous");
  if (contiguous != 1 || note_device(t, "workspace") || method_int(t, s_numel, &size) ||
      method_int(t, s_element_size, &item) || address(t, p))
    return -1;
  *bytes = (size_t)(size * item);
  return 0;
}

static PyObject* refused(const char* func, int rc) {
  PyObject* e = PyObject_CallFunction(c_error, "si", func, rc);
  if (e) {
    PyErr_SetObject(c_error, e);
    Py_DECREF(e);
  }
  return NULL;
}
static int count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 0;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
  return -1;
}
/* Fewer than the ABI's type holds: the library checks the rest. */
static int fits32(int64_t n, const char* name) {
  if (n <= INT32_MAX) return 0;
  PyErr_Format(PyExc_ValueError, "%s is too large", name);
  return -1;
}

/* ---- the calls -------------------------------------------------------------------- */

/* dims, q, k, q_norm, k_norm, inv_freq, positions, q_out, k_out, rope_scale, d_status,
   stream */
static PyObject* qk_norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_rope_params p;
  gdn_view q, k;
  PyObject *dt, *other;
  int64_t n;
  void *pos, *status, *qp = NULL, *kp = NULL;
  gdn_stream_t s;
  if (count(na, 12) || dims_of(a[0], &d, &dt) || method_int(a[6], s_numel, &n) ||
      view(a[1], "q", dt, n, d.h_q, d.d, &q) || view(a[2], "k", dt, n, d.h_kv, d.d, &k) ||
      rope_params(a + 3, &d, a[9], &p) || flat(a[6], "positions", t_int32, n, &pos) ||
      flat(a[10], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[11], &s, &other))
    return NULL;
  p.d_status = status;
  PyObject *qo = Py_NewRef(Py_None), *ko = Py_NewRef(Py_None), *r = NULL;
  if (a[1] != Py_None) Py_SETREF(qo, output(a[7], "q_out", dt, n, d.h_q, d.d, a[1], other, &qp));
  if (qo && a[2] != Py_None)
    Py_SETREF(ko, output(a[8], "k_out", dt, n, d.h_kv, d.d, a[2], other, &kp));
  if (qo && ko) {
    const int rc = call_norm_rope(&d, &p, &q, &k, pos, n, qp, kp, s);
    r = rc ? refused("gdn_qk_norm_rope", rc) : PyTuple_Pack(2, qo, ko);
  }
  Py_XDECREF(qo);
  Py_XDECREF(ko);
  return r;
}

/* dims, q, k, v, q_norm, k_norm, inv_freq, positions, k_cache, v_cache, block_table,
   row_seq, q_out, k_out, rope_scale, d_status, stream */
static PyObject* kv_append(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_rope_params p;
  gdn_view q, k, v;
  gdn_kv_cache c;
  PyObject *dt, *other;
  int64_t n;
  void *pos, *seq, *status, *qp = NULL, *kp;
  gdn_stream_t s;
  if (count(na, 17) || dims_of(a[0], &d, &dt) || method_int(a[7], s_numel, &n) ||
      view(a[1], "q", dt, n, d.h_q, d.d, &q) || view(a[2], "k", dt, n, d.h_kv, d.d, &k) ||
      view(a[3], "v", dt, n, d.h_kv, d.d, &v) || rope_params(a + 4, &d, a[14], &p) ||
      flat(a[7], "positions", t_int32, n, &pos) || cache_of(a + 8, &d, dt, &c) ||
      flat(a[11], "row_seq", t_int32, n, &seq) ||
      flat(a[13], "k_out", dt, n * d.h_kv * d.d, &kp) ||
      flat(a[15], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[16], &s, &other))
    return NULL;
  PyObject* qo = Py_NewRef(Py_None);
  if (a[1] != Py_None) Py_SETREF(qo, output(a[12], "q_out", dt, n, d.h_q, d.d, a[1], other, &qp));
  if (!qo) return NULL;
  const int rc = call_append(&d, &p, &q, &k, &v, pos, seq, n, &c, qp, kp, status, s);
  if (!rc) return qo;
  Py_DECREF(qo);
  return refused("gdn_kv_append", rc);
}

/* dims, q, k, v, cu_seqlens, cu_seqlens_kv, gate, o, d_status, stream */
static PyObject* attn_prefill(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_view q, k, v, gate;
  PyObject *dt, *other;
  int64_t ends, sq[4] = {0}, sk[4] = {0};
  void *cu, *cu_kv, *status, *op;
  gdn_stream_t s;
  if (count(na, 10) || dims_of(a[0], &d, &dt) || shape_of(a[1], sq) < 0 || shape_of(a[2], sk) < 0 ||
      method_int(a[4], s_numel, &ends) || view(a[1], "q", dt, sq[0], d.h_q, d.d, &q) ||
      view(a[2], "k", dt, sk[0], d.h_kv, d.d, &k) || view(a[3], "v", dt, sk[0], d.h_kv, d.d, &v) ||
      view(a[6], "gate", dt, sq[0], d.h_q, d.d, &gate) || fits32(ends, "cu_seqlens") ||
      flat(a[4], "cu_seqlens", t_int32, ends, &cu) ||
      flat(a[5], "cu_seqlens_kv", t_int32, ends, &cu_kv) ||
      flat(a[8], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[9], &s, &other))
    return NULL;
  PyObject* o = output(a[7], "o", dt, sq[0], d.h_q, d.d, a[1], other, &op);
  if (!o) return NULL;
  const int rc = call_prefill(&d, &q, &k, &v, cu, cu_kv, (int32_t)(ends - 1), sq[0], sk[0], &gate, op,
                              status, s);
  if (!rc) return o;
  Py_DECREF(o);
  return refused("gdn_attn_prefill", rc);
}

/* dims, q, k_cache, v_cache, block_table, seq_lens, workspace, shared_len, gate, o,
   d_status, stream */
static PyObject* attn_decode(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_view q, gate;
  gdn_kv_cache c;
  PyObject *dt, *other;
  int64_t sq[4] = {0};
  size_t size;
  void *lens, *status, *op, *ws;
  gdn_stream_t s;
  if (count(na, 12) || dims_of(a[0], &d, &dt) || shape_of(a[1], sq) < 0 || fits32(sq[0], "q") ||
      view(a[1], "q", dt, sq[0], d.h_q, d.d, &q) ||
      view(a[8], "gate", dt, sq[0], d.h_q, d.d, &gate) || cache_of(a + 2, &d, dt, &c) ||
      flat(a[5], "seq_lens", t_int32, sq[0], &lens) ||
      flat(a[10], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[11], &s, &other))
    return NULL;
  const int64_t shared = PyLong_AsLongLong(a[7]);
  if (shared == -1 && PyErr_Occurred()) return NULL;
  if (workspace_of(a[6], &ws, &size) || all_device()) return NULL;
  PyObject* o = output(a[9], "o", dt, sq[0], d.h_q, d.d, a[1], other, &op);
  if (!o) return NULL;
  const int rc = call_decode(&d, &q, &c, lens, (int32_t)sq[0], shared, &gate, op, ws, size, status, s);
  if (!rc) return o;
  Py_DECREF(o);
  return refused("gdn_attn_decode", rc);
}

/* ---- positions with several axes, the 8-bit cache ---------------------------------- */

/* The axes of a gdn_rope_axes; None: null. */
static int axes_of(PyObject* o, gdn_rope_axes* a, const gdn_rope_axes** p) {
  *p = NULL;
  if (o == Py_None) return 0;
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) return -1;
  const int fits = b.len == (Py_ssize_t)sizeof(*a);
  if (fits) memcpy(a, b.buf, sizeof(*a));
  PyBuffer_Release(&b);
  if (!fits) {
    PyErr_SetString(PyExc_TypeError, "axes must be a gdn_rope_axes");
    return -1;
  }
  *p = a;
  return 0;
}
/* How many positions each of n tokens has. */
static int64_t per_token(const gdn_rope_axes* a) {
  return a && a->count >= 0 && a->count <= GDN_ROPE_MAX_AXES ? a->count : 1;
}

/* What a Kv8Cache keeps of its tensors, looked at once when it is made. */
typedef struct {
  gdn_kv8_cache c;
  int64_t h_kv, page_size, d, device;
} kv8_handle;

/* k, v, k_scale, v_scale, block_table -> the handle, as bytes */
static PyObject* kv8_make(PyObject* self, PyObject* const* t, Py_ssize_t na) {
  (void)self;
  kv8_handle h;
  memset(&h, 0, sizeof(h));
  host_tensor = odd_tensor = NULL;
  call_device = -1;
  if (count(na, 5)) return NULL;
  int64_t k[4], b[4];
  const int nk = shape_of(t[0], k);
  if (nk < 0) return NULL;
  if (nk != 4 || k[2] % GDN_KV8_BLOCK) {
    PyErr_Format(PyExc_ValueError, "k must be [num_pages, h_kv, page_size, d], pages of whole blocks of %d",
                 GDN_KV8_BLOCK);
    return NULL;
  }
  const int nb = shape_of(t[4], b);
  if (nb < 0) return NULL;
  if (nb != 2 || b[0] > INT32_MAX || b[1] > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "block_table must be [num_seqs, pages_per_seq]");
    return NULL;
  }
  const int64_t rows = k[0] * k[1] * k[2], scales = rows / GDN_KV8_BLOCK;
  void *ks, *vs, *table;
  if (flat(t[0], "k", t_e4m3, rows * k[3], &h.c.k) || flat(t[1], "v", t_e4m3, rows * k[3], &h.c.v) ||
      flat(t[2], "k_scale", io_types[GDN_FP32], scales, &ks) ||
      flat(t[3], "v_scale", io_types[GDN_FP32], scales, &vs) ||
      flat(t[4], "block_table", t_int32, b[0] * b[1], &table))
    return NULL;
  if (odd_tensor || (host_tensor && call_device >= 0)) {
    PyErr_Format(PyExc_ValueError, "a cache's tensors must be on one device");
    return NULL;
  }
  h.c.k_scale = ks;
  h.c.v_scale = vs;
  h.c.block_table = table;
  h.c.num_pages = k[0];
  h.c.num_seqs = (int32_t)b[0];
  h.c.pages_per_seq = (int32_t)b[1];
  h.h_kv = k[1];
  h.page_size = k[2];
  h.d = k[3];
  h.device = call_device;
  return PyBytes_FromStringAndSize((const char*)&h, sizeof(h));
}

/* A Kv8Cache, by its handle. */
static int kv8_of(PyObject* o, const char* name, const gdn_attn_dims* d, gdn_kv8_cache* c) {
  PyObject* b = PyObject_GetAttr(o, s_handle);
  if (!b || !PyBytes_Check(b) || PyBytes_GET_SIZE(b) != (Py_ssize_t)sizeof(kv8_handle)) {
    Py_XDECREF(b);
    PyErr_Format(PyExc_TypeError, "%s must be a Kv8Cache", name);
    return -1;
  }
  kv8_handle h;
  memcpy(&h, PyBytes_AS_STRING(b), sizeof(h));
  Py_DECREF(b);
  /* its tensors are where they were when it was made */
  const void* made[5] = {h.c.k, h.c.v, h.c.k_scale, h.c.v_scale, h.c.block_table};
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) {
    PyErr_Format(PyExc_TypeError, "%s must be a Kv8Cache", name);
    return -1;
  }
  for (int i = 0; i < 5; ++i) {
    void* now;
    if (address(PyTuple_GET_ITEM(o, i), &now)) return -1;
    if (now != made[i]) {
      PyErr_Format(PyExc_ValueError, "%s has a tensor whose memory is another than when it was made",
                   name);
      return -1;
    }
  }
  if (h.h_kv != d->h_kv || h.page_size != d->page_size || h.d != d->d) {
    PyErr_Format(PyExc_ValueError, "%s.k must be [num_pages, %d, %d, %d]", name, d->h_kv,
                 d->page_size, d->d);
    return -1;
  }
  *c = h.c;
  if (h.device < 0) {
    if (!host_tensor) host_tensor = name;
  } else if (call_device < 0) {
    call_device = h.device;
  } else if (h.device != call_device && !odd_tensor) {
    odd_tensor = name;
    odd_device = h.device;
  }
  return 0;
}
/* An integer argument that the ABI takes in 32 bits. */
static int int32_of(PyObject* o, const char* name, int32_t* out) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (v > INT32_MAX || v < INT32_MIN) {
    PyErr_Format(PyExc_ValueError, "%s does not fit in 32 bits", name);
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

/* dims, q, k, q_norm, k_norm, inv_freq, positions, axes, q_out, k_out, rope_scale,
   d_status, stream */
static PyObject* qk_norm_rope_axes(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_rope_params p;
  gdn_rope_axes axes;
  const gdn_rope_axes* ax;
  gdn_view q, k;
  PyObject *dt, *other;
  int64_t total, rows[4] = {0};
  void *pos, *status, *qp = NULL, *kp = NULL;
  gdn_stream_t s;
  if (count(na, 13) || dims_of(a[0], &d, &dt) || axes_of(a[7], &axes, &ax) ||
      method_int(a[6], s_numel, &total))
    return NULL;
  if (!ax) {
    PyErr_SetString(PyExc_TypeError, "axes must be a gdn_rope_axes");
    return NULL;
  }
  /* as many tokens as q or k has: where the axes are not as many as the positions', those are at fault */
  PyObject* const some = a[1] != Py_None ? a[1] : a[2];
  if (some != Py_None && shape_of(some, rows) < 0) return NULL;
  const int64_t n = some != Py_None ? rows[0] : per_token(ax) ? total / per_token(ax) : 0;
  if (view(a[1], "q", dt, n, d.h_q, d.d, &q) || view(a[2], "k", dt, n, d.h_kv, d.d, &k) ||
      rope_params(a + 3, &d, a[10], &p) ||
      flat(a[6], "positions", t_int32, n * per_token(ax), &pos) ||
      flat(a[11], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[12], &s, &other))
    return NULL;
  p.d_status = status;
  PyObject *qo = Py_NewRef(Py_None), *ko = Py_NewRef(Py_None), *r = NULL;
  if (a[1] != Py_None) Py_SETREF(qo, output(a[8], "q_out", dt, n, d.h_q, d.d, a[1], other, &qp));
  if (qo && a[2] != Py_None)
    Py_SETREF(ko, output(a[9], "k_out", dt, n, d.h_kv, d.d, a[2], other, &kp));
  if (qo && ko) {
    const int rc = call_norm_rope_axes(&d, &p, ax, &q, &k, pos, n, qp, kp, s);
    r = rc ? refused("gdn_qk_norm_rope_axes", rc) : PyTuple_Pack(2, qo, ko);
  }
  Py_XDECREF(qo);
  Py_XDECREF(ko);
  return r;
}

/* dims, q, k, v, q_norm, k_norm, inv_freq, positions, cache, starts, cu_seqlens, axes,
   q_out, k_out, rope_scale, d_status, stream */
static PyObject* kv8_append(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_rope_params p;
  gdn_rope_axes axes;
  const gdn_rope_axes* ax;
  gdn_view q, k, v;
  gdn_kv8_cache c;
  PyObject *dt, *other;
  int64_t sk[4] = {0}, seqs;
  void *pos, *starts, *cu, *status, *qp = NULL, *kp;
  gdn_stream_t s;
  if (count(na, 17) || dims_of(a[0], &d, &dt) || axes_of(a[11], &axes, &ax) ||
      shape_of(a[2], sk) < 0 || method_int(a[9], s_numel, &seqs) || fits32(seqs, "starts"))
    return NULL;
  const int64_t n = sk[0];
  if (view(a[1], "q", dt, n, d.h_q, d.d, &q) || view(a[2], "k", dt, n, d.h_kv, d.d, &k) ||
      view(a[3], "v", dt, n, d.h_kv, d.d, &v) || rope_params(a + 4, &d, a[14], &p) ||
      flat(a[7], "positions", t_int32, n * per_token(ax), &pos) || kv8_of(a[8], "cache", &d, &c) ||
      flat(a[9], "starts", t_int32, seqs, &starts) ||
      flat(a[10], "cu_seqlens", t_int32, seqs + 1, &cu) ||
      flat(a[13], "k_out", dt, n * d.h_kv * d.d, &kp) ||
      flat(a[15], "d_status", t_int32, 1, &status) || all_device() ||
      stream_of(a[16], &s, &other))
    return NULL;
  PyObject* qo = Py_NewRef(Py_None);
  if (a[1] != Py_None) Py_SETREF(qo, output(a[12], "q_out", dt, n, d.h_q, d.d, a[1], other, &qp));
  if (!qo) return NULL;
  const int rc = call_kv8_append(&d, &p, ax, &q, &k, &v, pos, cu, starts, (int32_t)seqs, n, &c, qp, kp,
                                 status, s);
  if (!rc) return qo;
  Py_DECREF(qo);
  return refused("gdn_kv8_append", rc);
}

/* dims, cache, cu_seqlens, total, k_out, v_out, d_status, stream */
static PyObject* kv8_gather(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_kv8_cache c;
  PyObject *dt, *other;
  int64_t ends;
  void *cu, *status, *kp, *vp;
  gdn_stream_t s;
  if (count(na, 8) || dims_of(a[0], &d, &dt) || kv8_of(a[1], "cache", &d, &c) ||
      method_int(a[2], s_numel, &ends) || fits32(ends, "cu_seqlens") ||
      flat(a[2], "cu_seqlens", t_int32, ends, &cu) ||
      flat(a[6], "d_status", t_int32, 1, &status) || all_device() || stream_of(a[7], &s, &other))
    return NULL;
  const int64_t total = PyLong_AsLongLong(a[3]);
  if (total == -1 && PyErr_Occurred()) return NULL;
  const int64_t rows = total > 0 ? total : 0;   /* the library refuses less */
  PyObject* like = a[2];
  PyObject *r = NULL, *vo = NULL, *ko = output(a[4], "k_out", dt, rows, d.h_kv, d.d, like, other, &kp);
  if (ko) vo = output(a[5], "v_out", dt, rows, d.h_kv, d.d, like, other, &vp);
  if (vo) {
    const int rc = call_kv8_gather(&d, &c, cu, (int32_t)(ends - 1), total, kp, vp, status, s);
    r = rc ? refused("gdn_kv8_gather", rc) : PyTuple_Pack(2, ko, vo);
  }
  Py_XDECREF(ko);
  Py_XDECREF(vo);
  return r;
}

/* dims, q, cache, seq_lens, workspace, gate, weights, o, d_status, stream */
static PyObject* attn_decode_kv8(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_view q, gate;
  gdn_kv8_cache c;
  PyObject *dt, *other;
  int64_t sq[4] = {0};
  size_t size;
  void *lens, *weights, *status, *op, *ws;
  gdn_stream_t s;
  if (count(na, 10) || dims_of(a[0], &d, &dt) || shape_of(a[1], sq) < 0 || fits32(sq[0], "q") ||
      view(a[1], "q", dt, sq[0], d.h_q, d.d, &q) || kv8_of(a[2], "cache", &d, &c) ||
      view(a[5], "gate", dt, sq[0], d.h_q, d.d, &gate) ||
      flat(a[3], "seq_lens", t_int32, sq[0], &lens) ||
      flat(a[6], "weights", io_types[GDN_FP32],
           (int64_t)c.num_seqs * d.h_kv * c.pages_per_seq * d.page_size, &weights) ||
      flat(a[8], "d_status", t_int32, 1, &status) || workspace_of(a[4], &ws, &size) ||
      all_device() || stream_of(a[9], &s, &other))
    return NULL;
  PyObject* o = output(a[7], "o", dt, sq[0], d.h_q, d.d, a[1], other, &op);
  if (!o) return NULL;
  const int rc =
      call_decode_kv8(&d, &q, &c, lens, (int32_t)sq[0], &gate, weights, op, ws, size, status, s);
  if (!rc) return o;
  Py_DECREF(o);
  return refused("gdn_attn_decode_kv8", rc);
}

/* dims, from, weights, seq_lens, keep, to, weights_out, first, last, new_lens, kept,
   d_status, stream */
static PyObject* kv8_evict(PyObject* self, PyObject* const* a, Py_ssize_t na) {
  (void)self;
  gdn_attn_dims d;
  gdn_kv8_cache c, to;
  PyObject *dt, *other;
  int64_t n;
  int32_t keep, first, last;
  void *weights, *lens, *out, *status, *np, *kp;
  gdn_stream_t s;
  if (count(na, 13) || dims_of(a[0], &d, &dt) || kv8_of(a[1], "cache", &d, &c) ||
      kv8_of(a[5], "to", &d, &to) || method_int(a[3], s_numel, &n) || fits32(n, "seq_lens") ||
      flat(a[2], "weights", io_types[GDN_FP32],
           (int64_t)c.num_seqs * d.h_kv * c.pages_per_seq * d.page_size, &weights) ||
      flat(a[6], "weights_out", io_types[GDN_FP32],
           (int64_t)to.num_seqs * d.h_kv * to.pages_per_seq * d.page_size, &out) ||
      flat(a[3], "seq_lens", t_int32, n, &lens) || int32_of(a[4], "keep", &keep) ||
      int32_of(a[7], "first", &first) || int32_of(a[8], "last", &last) ||
      flat(a[11], "d_status", t_int32, 1, &status) || all_device() || stream_of(a[12], &s, &other))
    return NULL;
  const int64_t rows = keep > 0 ? keep : 0;   /* the library refuses less */
  PyObject *r = NULL, *ko = NULL, *size = Py_BuildValue("(L)", (long long)n);
  PyObject* no = shaped(a[9], "new_lens", t_int32, size, n, a[3], other, &np);
  Py_XDECREF(size);
  if (no) ko = output(a[10], "kept", t_int32, n, d.h_kv, rows, a[3], other, &kp);
  if (ko) {
    const int rc = call_kv8_evict(&d, &c, weights, lens, (int32_t)n, keep, first, last, &to, out, np, kp,
                                  status, s);
    r = rc ? refused("gdn_kv8_evict", rc) : PyTuple_Pack(2, no, ko);
  }
  Py_XDECREF(no);
  Py_XDECREF(ko);
  return r;
}

/* After setup: float8_e4m3fn, the entry points' addresses. */
static PyObject* setup_kv8(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long fn[5];
  if (!PyArg_ParseTuple(args, "O(KKKKK)", &t_e4m3, &fn[0], &fn[1], &fn[2], &fn[3], &fn[4]))
    return NULL;
  Py_INCREF(t_e4m3);
  call_norm_rope_axes = (norm_rope_axes_fn)(uintptr_t)fn[0];
  call_kv8_append = (kv8_append_fn)(uintptr_t)fn[1];
  call_kv8_gather = (kv8_gather_fn)(uintptr_t)fn[2];
  call_decode_kv8 = (decode_kv8_fn)(uintptr_t)fn[3];
  call_kv8_evict = (kv8_evict_fn)(uintptr_t)fn[4];
  Py_RETURN_NONE;
}

/* (float32, bfloat16, float16), int32, float64, torch.empty, empty(size, dtype, device,
   stream), current raw stream of a device, current device, GdnError, the four entry
   points' addresses */
static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long fn[4];
  if (!PyArg_ParseTuple(args, "(OOO)OOOOOOO(KKKK)", &io_types[0], &io_types[1], &io_types[2],
                        &t_int32, &t_float64, &f_empty, &f_empty_on, &f_stream, &f_device, &c_error,
                        &fn[0], &fn[1], &fn[2], &fn[3]))
    return NULL;
  for (int i = 0; i < 3; ++i) Py_INCREF(io_types[i]);
  Py_INCREF(t_int32);
  Py_INCREF(t_float64);
  Py_INCREF(f_empty);
  Py_INCREF(f_empty_on);
  Py_INCREF(f_stream);
  Py_INCREF(f_device);
  Py_INCREF(c_error);
  call_norm_rope = (norm_rope_fn)(uintptr_t)fn[0];
  call_append = (append_fn)(uintptr_t)fn[1];
  call_prefill = (prefill_fn)(uintptr_t)fn[2];
  call_decode = (decode_fn)(uintptr_t)fn[3];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, NULL},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, NULL},
    {"attn_prefill", (PyCFunction)(void (*)(void))attn_prefill, METH_FASTCALL, NULL},
    {"attn_decode", (PyCFunction)(void (*)(void))attn_decode, METH_FASTCALL, NULL},
    {"setup_kv8", setup_kv8, METH_VARARGS, NULL},
    {"kv8_make", (PyCFunction)(void (*)(void))kv8_make, METH_FASTCALL, NULL},
    {"qk_norm_rope_axes", (PyCFunction)(void (*)(void))qk_norm_rope_axes, METH_FASTCALL, NULL},
    {"kv8_append", (PyCFunction)(void (*)(void))kv8_append, METH_FASTCALL, NULL},
    {"kv8_gather", (PyCFunction)(void (*)(void))kv8_gather, METH_FASTCALL, NULL},
    {"attn_decode_kv8", (PyCFunction)(void (*)(void))attn_decode_kv8, METH_FASTCALL, NULL},
    {"kv8_evict", (PyCFunction)(void (*)(void))kv8_evict, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_calls",
                                    "Marshalling of the full-attention calls.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__attn_calls(void) {
  struct {
    PyObject** at;
    const char* name;
  } names[] = {{&s_shape, "shape"},   {&s_stride, "stride"}, {&s_dtype, "dtype"},
               {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},   {&s_is_contiguous, "is_contiguous"},
               {&s_device, "device"}, {&s_get_device, "get_device"},
               {&s_element_size, "element_size"}, {&s_handle, "handle"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].at = PyUnicode_InternFromString(names[i].name))) return NULL;
  if (!(empty_kw = Py_BuildValue("(ss)", "dtype", "device"))) return NULL;
  return PyModule_Create(&module);
}
