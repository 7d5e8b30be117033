/*
 * The binding of the 16-bit operators, whose calls may be shorter than their
 * marshalling: one token's layer norm runs 2.5 us on the device, and a ctypes
 * call with its checks in Python took 4.7 us of the host beside the launch;
 * this takes about 1.5.  Argument marshalling and checks only; the work is
 * libsvdq.so's.  Uses the CPython API and the tensors' Python attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "svdq.h"

static PyObject *s_shape, *s_dtype, *s_stride, *s_data_ptr, *s_get_device, *s_is_contiguous, *s_nbytes;
static PyObject *g_dtypes[3];              /* torch.bfloat16, .float16, .float32 */
static PyObject *g_int32, *g_device, *g_raw_stream;

typedef struct {
  int ndim;
  long long shape[3], stride[3];
  void *ptr;
  int dev;
  int code;                                /* SVDQ_DTYPE_*, 3: torch.int32, -1: another type */
} Tensor;

/* A tuple of 1 to 3 integers. */
static int read_tuple(PyObject *t, long long *out, const char *name) {
  Py_ssize_t n, i;
  if (!PyTuple_Check(t) || (n = PyTuple_GET_SIZE(t)) < 1 || n > 3) {
    PyErr_Format(PyExc_ValueError, "%s: expected a tensor of 1 to 3 dimensions", name);
    return -1;
  }
  for (i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    if (out[i] == -1 && PyErr_Occurred()) return -1;
  }
  return (int)n;
}

static int read_tensor(PyObject *o, const char *name, Tensor *t) {
  PyObject *v;
  if (!(v = PyObject_GetAttr(o, s_shape))) return -1;
  t->ndim = read_tuple(v, t->shape, name);
  Py_DECREF(v);
  if (t->ndim < 0) return -1;
  if (!(v = PyObject_CallMethodNoArgs(o, s_stride))) return -1;
  const int n = read_tuple(v, t->stride, name);
  Py_DECREF(v);
  if (n < 0) return -1;
  if (!(v = PyObject_GetAttr(o, s_dtype))) return -1;
  t->code = v == g_dtypes[0] ? 0 : v == g_dtypes[1] ? 1 : v == g_dtypes[2] ? 2 : v == g_int32 ? 3 : -1;
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(o, s_get_device))) return -1;
  t->dev = (int)PyLong_AsLong(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (!(v = PyObject_CallMethodNoArgs(o, s_data_ptr))) return -1;
  t->ptr = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

/* The element type of the call's first tensor, one of three. */
static int check_dtype(const Tensor *t, const char *name) {
  if (t->code < 0 || t->code > 2) {
    PyErr_Format(PyExc_ValueError, "%s: this dtype is not supported", name);
    return -1;
  }
  return 0;
}

/* The stream's handle; None: the current stream of device `dev`, which has to
 * be the current device (launches go there). */
static int read_stream(PyObject *o, int dev, cudaStream_t *st) {
  if (dev < 0) {
    PyErr_SetString(PyExc_ValueError, "the tensors have to be on a CUDA device");
    return -1;
  }
  PyObject *v = PyObject_CallNoArgs(g_device);
  if (!v) return -1;
  const long cur = PyLong_AsLong(v);
  if (cur != dev) {
    Py_DECREF(v);
    if (!PyErr_Occurred())
      PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, which is not the current device", dev);
    return -1;
  }
  if (o == Py_None) {
    PyObject *r = PyObject_CallOneArg(g_raw_stream, v);
    Py_DECREF(v);
    if (!r) return -1;
    *st = (cudaStream_t)PyLong_AsVoidPtr(r);
    Py_DECREF(r);
  } else {
    Py_DECREF(v);
    *st = (cudaStream_t)PyLong_AsVoidPtr(o);
  }
  return PyErr_Occurred() ? -1 : 0;
}

/* An epilogue as the C calls take it: what is no int is none of them (-1). */
static int read_epilogue(PyObject *o, int *epi) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return -1;
  *epi = v == (int)v ? (int)v : -1;
  return 0;
}

/* A leading dimension as the C calls take it. */
static int pitch(long long v) { return v < -0x7FFFFFFFll || v > 0x7FFFFFFFll ? -1 : (int)v; }

/* Pointer and leading dimension of a [rows, cols] tensor like X; None: null. */
static int read_matrix(PyObject *o, const char *name, long long rows, long long cols, const Tensor *x,
                       void **ptr, int *ld) {
  Tensor t;
  *ptr = NULL;
  *ld = 0;
  if (o == Py_None) return 0;
  if (read_tensor(o, name, &t) < 0) return -1;
  if (t.ndim != 2 || t.shape[0] != rows || t.shape[1] != cols) {
    PyErr_Format(PyExc_ValueError, "%s: expected shape (%lld, %lld)", name, rows, cols);
    return -1;
  }
  if (t.code != x->code || t.dev != x->dev) {
    PyErr_Format(PyExc_ValueError, "%s: expected the first tensor's dtype and device", name);
    return -1;
  }
  if (cols > 1 && t.stride[1] != 1) {
    PyErr_Format(PyExc_ValueError, "%s: rows have to be contiguous", name);
    return -1;
  }
  *ptr = t.ptr;
  *ld = pitch(rows <= 1 ? (cols + 7) / 8 * 8 : t.stride[0]);      /* a single row has no pitch */
  return 0;
}

static int read_vector(PyObject *o, const char *name, long long n, int code, int dev, void **ptr) {
  Tensor t;
  *ptr = NULL;
  if (o == Py_None) return 0;
  if (read_tensor(o, name, &t) < 0) return -1;
  if (t.ndim != 1 || t.shape[0] != n || (n > 1 && t.stride[0] != 1)) {
    PyErr_Format(PyExc_ValueError, "%s: expected %lld contiguous values", name, n);
    return -1;
  }
  if (t.code != code || t.dev != dev) {
    PyErr_Format(PyExc_ValueError, "%s: unexpected dtype or device", name);
    return -1;
  }
  *ptr = t.ptr;
  return 0;
}

/* A parameter [K], [1, K] (shared by every group) or [groups, K]. */
static int read_param(PyObject *o, const char *name, long long groups, long long K, int dev, int *code,
                      void **ptr, int *ld) {
  Tensor t;
  *ptr = NULL;
  *ld = 0;
  if (o == Py_None) return 0;
  if (read_tensor(o, name, &t) < 0) return -1;
  const int last = t.ndim - 1;
  const long long rows = t.ndim == 2 ? t.shape[0] : 1;
  if (t.ndim > 2 || t.shape[last] != K || (rows != 1 && rows != groups)) {
    PyErr_Format(PyExc_ValueError, "%s: expected [%lld, %lld] or [%lld]", name, groups, K, K);
    return -1;
  }
  if (t.dev != dev || t.code < 0 || t.code > 2 || (*code >= 0 && t.code != *code) ||
      (K > 1 && t.stride[last] != 1)) {
    PyErr_Format(PyExc_ValueError, "%s: expected contiguous rows of one type on cuda:%d", name, dev);
    return -1;
  }
  *code = t.code;
  *ptr = t.ptr;
  *ld = rows == 1 ? 0 : pitch(t.stride[0]);
  return 0;
}

static int nargs_are(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments", want);
  return 0;
}

static int read_sizes(const Tensor *x, const char *name) {
  if (x->ndim != 2 || x->shape[0] > 0x7FFFFFFF || x->shape[1] > 0x7FFFFFFF) {
    PyErr_Format(PyExc_ValueError, "%s: expected two sizes below 2^31", name);
    return -1;
  }
  return 0;
}

/* linear16(X, W, Y, bias, residual, epilogue, preact, stream) -> status */
static PyObject *linear16(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Tensor x, w;
  void *xp, *wp, *yp, *b, *r, *p;
  int ldx, ldw, ldy, ldr, ldp, epi;
  cudaStream_t st;
  svdq_status rc;
  if (!nargs_are(n, 8) || read_tensor(a[0], "X", &x) < 0 || check_dtype(&x, "X") < 0 ||
      read_sizes(&x, "X") < 0 || read_stream(a[7], x.dev, &st) < 0 || read_tensor(a[1], "W", &w) < 0 ||
      read_sizes(&w, "W") < 0)
    return NULL;
  const long long M = x.shape[0], K = x.shape[1], N = w.shape[0];
  if (read_epilogue(a[5], &epi) < 0) return NULL;
  if (w.shape[1] != K || w.code != x.code || w.dev != x.dev || (K > 1 && (w.stride[1] != 1 || x.stride[1] != 1))) {
    PyErr_SetString(PyExc_ValueError, "X, W: expected [M, K] and [N, K] of one type and device with contiguous rows");
    return NULL;
  }
  xp = x.ptr;
  wp = w.ptr;
  ldx = pitch(M <= 1 ? (K + 7) / 8 * 8 : x.stride[0]);
  ldw = pitch(N <= 1 ? (K + 7) / 8 * 8 : w.stride[0]);
  if (a[2] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "Y: expected a tensor");
    return NULL;
  }
  if (read_matrix(a[2], "Y", M, N, &x, &yp, &ldy) < 0 ||
      read_vector(a[3], "bias", N, x.code, x.dev, &b) < 0 ||
      read_matrix(a[4], "residual", M, N, &x, &r, &ldr) < 0 ||
      read_matrix(a[6], "preact", M, N, &x, &p, &ldp) < 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = svdq_linear16(x.code, (int)M, (int)K, (int)N, xp, ldx, wp, ldw, b, r, ldr, epi, yp, ldy, p,
                     ldp, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* layer_norm(X, Y, weight, bias, eps, weight_offset, rows_per_group, mean, rstd, stream) -> status */
static PyObject *layer_norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Tensor x;
  void *yp, *w, *b, *mu, *rs;
  int ldx, ldy, ldw, ldb, pc = -1;
  cudaStream_t st;
  svdq_status rc;
  if (!nargs_are(n, 10) || read_tensor(a[0], "X", &x) < 0 || check_dtype(&x, "X") < 0 ||
      read_sizes(&x, "X") < 0 || read_stream(a[9], x.dev, &st) < 0)
    return NULL;
  const long long M = x.shape[0], K = x.shape[1];
  const double eps = PyFloat_AsDouble(a[4]), off = PyFloat_AsDouble(a[5]);
  const long long rpg = PyLong_AsLongLong(a[6]);
  if (PyErr_Occurred()) return NULL;
  if (rpg > 0x7FFFFFFF || rpg < -0x7FFFFFFF) {
    PyErr_SetString(PyExc_ValueError, "rows_per_group: expected less than 2^31");
    return NULL;
  }
  if (K > 1 && x.stride[1] != 1) {
    PyErr_SetString(PyExc_ValueError, "X: rows have to be contiguous");
    return NULL;
  }
  ldx = pitch(M <= 1 ? (K + 7) / 8 * 8 : x.stride[0]);
  const long long groups = rpg > 0 ? (M + rpg - 1) / rpg : 1;
  if (a[1] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "Y: expected a tensor");
    return NULL;
  }
  if (read_matrix(a[1], "Y", M, K, &x, &yp, &ldy) < 0 ||
      read_param(a[2], "weight", groups, K, x.dev, &pc, &w, &ldw) < 0 ||
      read_param(a[3], "bias", groups, K, x.dev, &pc, &b, &ldb) < 0 ||
      read_vector(a[7], "mean", M, SVDQ_DTYPE_F32, x.dev, &mu) < 0 ||
      read_vector(a[8], "rstd", M, SVDQ_DTYPE_F32, x.dev, &rs) < 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = svdq_layer_norm(x.code, pc < 0 ? x.code : pc, (int)M, (int)K, x.ptr, ldx, w, ldw, b, ldb,
                       (float)off, (int)rpg, (float)eps, yp, ldy, mu, rs, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* A workspace (contiguous, any type), or None. */
static int read_workspace(PyObject *o, int dev, void **ptr, size_t *bytes) {
  PyObject *v;
  *ptr = NULL;
  *bytes = 0;
  if (o == Py_None) return 0;
  if (!(v = PyObject_CallMethodNoArgs(o, s_get_device))) return -1;
  const long d = PyLong_AsLong(v);
  Py_DECREF(v);
  if (!(v = PyObject_CallMethodNoArgs(o, s_is_contiguous))) return -1;
  const int whole = PyObject_IsTrue(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) return -1;
  if (d != dev || !whole) {
    PyErr_Format(PyExc_ValueError, "workspace: expected a contiguous tensor on cuda:%d", dev);
    return -1;
  }
  if (!(v = PyObject_GetAttr(o, s_nbytes))) return -1;
  *bytes = PyLong_AsSize_t(v);
  Py_DECREF(v);
  if (PyErr_Occurred() || !(v = PyObject_CallMethodNoArgs(o, s_data_ptr))) return -1;
  *ptr = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

/* linear16_backward(dY, X, W, preact, dX, dW, dbias, workspace, epilogue, stream) -> status */
static PyObject *linear16_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Tensor d, t;
  void *x, *w, *p, *gx, *gw, *gb, *ws;
  int ldd, ldx, ldw, ldp, ldgx, ldgw, epi;
  size_t bytes;
  cudaStream_t st;
  svdq_status rc;
  if (!nargs_are(n, 10) || read_tensor(a[0], "dY", &d) < 0 || check_dtype(&d, "dY") < 0 ||
      read_sizes(&d, "dY") < 0 || read_stream(a[9], d.dev, &st) < 0)
    return NULL;
  const long long M = d.shape[0], N = d.shape[1];
  long long K = 1;                         /* only dbias is wanted */
  PyObject *const with_k = a[1] != Py_None ? a[1] : a[2];
  if (with_k != Py_None) {
    if (read_tensor(with_k, "X, W", &t) < 0 || read_sizes(&t, "X, W") < 0) return NULL;
    K = t.shape[1];
  }
  if (read_epilogue(a[8], &epi) < 0) return NULL;
  if (N > 1 && d.stride[1] != 1) {
    PyErr_SetString(PyExc_ValueError, "dY: rows have to be contiguous");
    return NULL;
  }
  ldd = pitch(M <= 1 ? (N + 7) / 8 * 8 : d.stride[0]);
  if (read_matrix(a[1], "X", M, K, &d, &x, &ldx) < 0 || read_matrix(a[2], "W", N, K, &d, &w, &ldw) < 0 ||
      read_matrix(a[3], "preact", M, N, &d, &p, &ldp) < 0 ||
      read_matrix(a[4], "dX", M, K, &d, &gx, &ldgx) < 0 ||
      read_matrix(a[5], "dW", N, K, &d, &gw, &ldgw) < 0 ||
      read_vector(a[6], "dbias", N, d.code, d.dev, &gb) < 0 ||
      read_workspace(a[7], d.dev, &ws, &bytes) < 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = svdq_linear16_backward(d.code, (int)M, (int)K, (int)N, d.ptr, ldd, x, ldx, w, ldw, p, ldp, epi,
                              gx, ldgx, gw, ldgw, gb, ws, bytes, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* layer_norm_backward(dY, X, mean, rstd, dX, weight, weight_offset, rows_per_group, dweight, dbias,
 *                     workspace, stream) -> status */
static PyObject *layer_norm_backward(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Tensor x;
  void *d, *mu, *rs, *gx, *w, *gw, *gb, *ws;
  int ldx, ldd, ldgx, ldw, ldgw, ldgb, pc = -1;
  size_t bytes;
  cudaStream_t st;
  svdq_status rc;
  if (!nargs_are(n, 12) || read_tensor(a[1], "X", &x) < 0 || check_dtype(&x, "X") < 0 ||
      read_sizes(&x, "X") < 0 || read_stream(a[11], x.dev, &st) < 0)
    return NULL;
  const long long M = x.shape[0], K = x.shape[1];
  const double off = PyFloat_AsDouble(a[6]);
  const long long rpg = PyLong_AsLongLong(a[7]);
  if (PyErr_Occurred()) return NULL;
  if (rpg > 0x7FFFFFFF || rpg < -0x7FFFFFFF) {
    PyErr_SetString(PyExc_ValueError, "rows_per_group: expected less than 2^31");
    return NULL;
  }
  if (K > 1 && x.stride[1] != 1) {
    PyErr_SetString(PyExc_ValueError, "X: rows have to be contiguous");
    return NULL;
  }
  ldx = pitch(M <= 1 ? (K + 7) / 8 * 8 : x.stride[0]);
  const long long groups = rpg > 0 ? (M + rpg - 1) / rpg : 1;
  if (a[0] == Py_None || a[2] == Py_None || a[3] == Py_None) {
    PyErr_SetString(PyExc_ValueError, "dY, mean and rstd: expected tensors");
    return NULL;
  }
  if (read_matrix(a[0], "dY", M, K, &x, &d, &ldd) < 0 ||
      read_vector(a[2], "mean", M, SVDQ_DTYPE_F32, x.dev, &mu) < 0 ||
      read_vector(a[3], "rstd", M, SVDQ_DTYPE_F32, x.dev, &rs) < 0 ||
      read_matrix(a[4], "dX", M, K, &x, &gx, &ldgx) < 0 ||
      read_param(a[5], "weight", groups, K, x.dev, &pc, &w, &ldw) < 0 ||
      read_param(a[8], "dweight", groups, K, x.dev, &pc, &gw, &ldgw) < 0 ||
      read_param(a[9], "dbias", groups, K, x.dev, &pc, &gb, &ldgb) < 0 ||
      read_workspace(a[10], x.dev, &ws, &bytes) < 0)
    return NULL;
  /* a gradient has a row per group: one row is all of them only for one group */
  if ((gw && ldgw == 0 && groups != 1) || (gb && ldgb == 0 && groups != 1)) {
    PyErr_Format(PyExc_ValueError, "dweight, dbias: expected %lld rows", groups);
    return NULL;
  }
  if (gw && ldgw == 0) ldgw = pitch((K + 7) / 8 * 8);
  if (gb && ldgb == 0) ldgb = pitch((K + 7) / 8 * 8);
  Py_BEGIN_ALLOW_THREADS
  rc = svdq_layer_norm_backward(x.code, pc < 0 ? x.code : pc, (int)M, (int)K, d, ldd, x.ptr, ldx, mu, rs, w,
                                ldw, (float)off, (int)rpg, gx, ldgx, gw, ldgw, gb, ldgb, ws, bytes, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* rope(plan handle, axes, positions, X, out, inverse, stream) -> status */
static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  Tensor p, x, y;
  cudaStream_t st;
  svdq_status rc;
  int i;
  if (!nargs_are(n, 7)) return NULL;
  const svdq_rope_plan *plan = (const svdq_rope_plan *)PyLong_AsVoidPtr(a[0]);
  const long long axes = PyLong_AsLongLong(a[1]);
  const int inverse = PyObject_IsTrue(a[5]);
  if (PyErr_Occurred() || read_tensor(a[3], "X", &x) < 0 || check_dtype(&x, "X") < 0 ||
      read_tensor(a[4], "out", &y) < 0 || read_tensor(a[2], "positions", &p) < 0)
    return NULL;
  for (i = 0; i < 3; ++i)
    if (x.ndim != 3 || y.ndim != 3 || x.shape[i] != y.shape[i] || x.shape[i] > 0x7FFFFFFF) {
      PyErr_SetString(PyExc_ValueError, "X and out: expected [tokens, heads, head_dim]");
      return NULL;
    }
  if (y.code != x.code || y.dev != x.dev || (x.shape[2] > 1 && (x.stride[2] != 1 || y.stride[2] != 1))) {
    PyErr_SetString(PyExc_ValueError,
                    "X and out: expected one type and device and contiguous elements of a head");
    return NULL;
  }
  if (p.ndim != 2 || p.shape[1] != axes || p.shape[0] > 0x7FFFFFFF || p.code != 3 || p.dev != x.dev ||
      (axes > 1 && p.stride[1] != 1)) {
    PyErr_Format(PyExc_ValueError, "positions: expected int32 [rows, %lld] on the device of X", axes);
    return NULL;
  }
  if (read_stream(a[6], x.dev, &st) < 0) return NULL;
  Py_BEGIN_ALLOW_THREADS
  rc = svdq_rope(plan, x.code, (int)x.shape[0], (int)x.shape[1], (int)x.shape[2],
                 (const int32_t *)p.ptr, (int)p.shape[0], pitch(p.shape[0] > 1 ? p.stride[0] : axes),
                 x.ptr, x.stride[0], x.stride[1], y.ptr, y.stride[0], y.stride[1], inverse, st);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(rc);
}

/* init((bfloat16, float16, float32), int32, current device, current raw stream of a device) */
static PyObject *init(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int i;
  if (!nargs_are(n, 4) || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != 3) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "expected three dtypes");
    return NULL;
  }
  for (i = 0; i < 3; ++i) Py_XSETREF(g_dtypes[i], Py_NewRef(PyTuple_GET_ITEM(a[0], i)));
  Py_XSETREF(g_int32, Py_NewRef(a[1]));
  Py_XSETREF(g_device, Py_NewRef(a[2]));
  Py_XSETREF(g_raw_stream, Py_NewRef(a[3]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"linear16", (PyCFunction)(void (*)(void))linear16, METH_FASTCALL, NULL},
    {"linear16_backward", (PyCFunction)(void (*)(void))linear16_backward, METH_FASTCALL, NULL},
    {"layer_norm_backward", (PyCFunction)(void (*)(void))layer_norm_backward, METH_FASTCALL, NULL},
    {"layer_norm", (PyCFunction)(void (*)(void))layer_norm, METH_FASTCALL, NULL},
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_svdq_fastcall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__svdq_fastcall(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  if (!s_is_contiguous || !s_nbytes || !s_shape || !s_dtype || !s_stride || !s_data_ptr || !s_get_device) return NULL;
  return PyModule_Create(&module);
}
