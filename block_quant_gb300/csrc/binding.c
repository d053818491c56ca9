/* Argument marshalling of the layer operators for Python (CPython C API, no torch
 * headers): reads pointer, shape, pitch and type off torch tensors, packs them as
 * bq_call takes them and calls it.  A generated token's norm costs a few
 * microseconds in all; reading its seven tensors from Python code took most of them.
 *
 * Matrices are 2-D tensors whose rows are contiguous, vectors contiguous 1-D ones.
 * Each function returns bq_call's code, or raises ValueError for an argument of the
 * wrong type or shape (the package turns it into its own error). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

enum { BF16 = 1, FP32 = 2, FP8 = 4 }; /* what an argument may be: 1 << BQ_ROWS_* */

static int (*g_call)(int, const void*);
static PyObject *g_kinds;                 /* torch dtype -> kind (0, 1, 2); 32, 64: id types */
static PyObject *g_fill;                  /* called with an unknown dtype: its kind or None */
static PyObject *g_current;               /* called without arguments: the current device */
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_get_device, *s_nbytes;

typedef struct {
  int64_t p, ld, rows, cols, kind;
} Mat;

static int64_t kind_of(PyObject* x, const char* name) {
  PyObject* d = PyObject_GetAttr(x, s_dtype);
  if (!d) return -1;
  PyObject* k = PyDict_GetItemWithError(g_kinds, d);
  if (!k && !PyErr_Occurred()) {
    PyObject* v = PyObject_CallOneArg(g_fill, d);
    if (v && v != Py_None && PyDict_SetItem(g_kinds, d, v) == 0) k = v; /* the dict holds it */
    Py_XDECREF(v);
    if (!k && !PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s has type %S", name, d);
  }
  Py_DECREF(d);
  return k ? PyLong_AsLongLong(k) : -1;
}

/* the tensor's address; all of a call's tensors must be on one GPU: *dev, -1 before the first
 * (each call's own: Python code that runs in between may make other calls) */
static int pointer_of(int64_t* dev, PyObject* x, const char* name, int64_t* p) {
  PyObject* v = PyObject_CallMethodNoArgs(x, s_get_device);
  if (!v) return -1;
  const int64_t d = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (d < 0 || (*dev >= 0 && d != *dev)) {
    if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, d < 0 ? "%s is not on a GPU" : "%s is on another GPU", name);
    return -1;
  }
  *dev = d;
  v = PyObject_CallMethodNoArgs(x, s_data_ptr);
  if (!v) return -1;
  *p = (int64_t)PyLong_AsUnsignedLongLong(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

/* n values of a tuple of exactly n integers */
static int ints(PyObject* t, int n, int64_t* v, const char* name) {
  if (!t) return -1;
  int ok = PyTuple_Check(t) && PyTuple_GET_SIZE(t) == n;
  for (int i = 0; ok && i < n; ++i) v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  Py_DECREF(t);
  if (!ok) PyErr_Format(PyExc_ValueError, "%s must have %d dimension%s", name, n, n == 1 ? "" : "s");
  return ok && !PyErr_Occurred() ? 0 : -1;
}

/* rows, columns and pitch of a 2-D tensor with contiguous rows; rows, cols: -1 for any */
static int shape_of(PyObject* x, const char* name, int64_t rows, int64_t cols, Mat* m) {
  int64_t s[2], st[2];
  if (ints(PyObject_GetAttr(x, s_shape), 2, s, name) || ints(PyObject_CallMethodNoArgs(x, s_stride), 2, st, name)) return -1;
  if ((rows >= 0 && s[0] != rows) || (cols >= 0 && s[1] != cols)) {
    PyErr_Format(PyExc_ValueError, "%s is %lld x %lld, expected %lld x %lld (-1: any)", name, (long long)s[0],
                 (long long)s[1], (long long)rows, (long long)cols);
    return -1;
  }
  if (st[1] != 1 && s[1] > 1) {
    PyErr_Format(PyExc_ValueError, "%s's rows must be contiguous", name);
    return -1;
  }
  m->ld = st[0], m->rows = s[0], m->cols = s[1];
  return 0;
}

/* rows, cols: -1 for any */
static int mat(int64_t* dev, PyObject* x, const char* name, int kinds, int64_t rows, int64_t cols, Mat* m) {
  if (x == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s is None", name);
    return -1;
  }
  m->kind = kind_of(x, name);
  if (m->kind < 0) return -1;
  if (m->kind > 2 || !(kinds >> m->kind & 1)) {
    PyErr_Format(PyExc_ValueError, "%s has a type that is not taken", name);
    return -1;
  }
  return shape_of(x, name, rows, cols, m) ? -1 : pointer_of(dev, x, name, &m->p);
}

/* a matrix that may be None: zeros */
static int opt(int64_t* dev, PyObject* x, const char* name, int kinds, int64_t rows, int64_t cols, Mat* m) {
  memset(m, 0, sizeof *m);
  return x == Py_None ? 0 : mat(dev, x, name, kinds, rows, cols, m);
}

static int contiguous(PyObject* x, const char* name) {
  PyObject* v = PyObject_CallMethodNoArgs(x, s_is_contiguous);
  if (!v) return -1;
  const int ok = v == Py_True;
  Py_DECREF(v);
  if (!ok) PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
  return ok ? 0 : -1;
}

/* a matrix of ids (int32 or int64): m->kind their bits */
static int id_mat(int64_t* dev, PyObject* x, const char* name, int64_t rows, int64_t cols, Mat* m) {
  if (x == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s is None", name);
    return -1;
  }
  const int64_t k = kind_of(x, name);
  if (k < 0) return -1;
  if (k != 32 && k != 64) {
    PyErr_Format(PyExc_ValueError, "%s has a type that is not taken", name);
    return -1;
  }
  if (shape_of(x, name, rows, cols, m)) return -1;
  m->kind = k;
  return pointer_of(dev, x, name, &m->p);
}

/* n: -1 for any; returns the length in *got */
static int vec(int64_t* dev, PyObject* x, const char* name, int kinds, int64_t n, int64_t* p, int64_t* kind, int64_t* got) {
  if (x == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s is None", name);
    return -1;
  }
  int64_t k = kind_of(x, name), len;
  if (k < 0) return -1;
  if (kinds == 0 ? (k != 32 && k != 64) : (k > 2 || !(kinds >> k & 1))) {
    PyErr_Format(PyExc_ValueError, "%s has a type that is not taken", name);
    return -1;
  }
  if (ints(PyObject_GetAttr(x, s_shape), 1, &len, name) || contiguous(x, name)) return -1;
  if (n >= 0 && len != n) {
    PyErr_Format(PyExc_ValueError, "%s has %lld values, expected %lld", name, (long long)len, (long long)n);
    return -1;
  }
  if (kind) *kind = k;
  if (got) *got = len;
  return pointer_of(dev, x, name, p);
}

/* one fp32 scale per 128 x 128 tile, contiguous, of any shape */
static int tiles(int64_t* dev, PyObject* x, const char* name, int64_t rows, int64_t cols, int64_t* p) {
  if (x == Py_None) {
    PyErr_Format(PyExc_ValueError, "%s is None", name);
    return -1;
  }
  const int64_t k = kind_of(x, name);
  if (k < 0) return -1;
  PyObject* t = PyObject_GetAttr(x, s_shape);
  if (!t) return -1;
  int64_t n = 1;
  for (Py_ssize_t i = 0; PyTuple_Check(t) && i < PyTuple_GET_SIZE(t); ++i) n *= PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  Py_DECREF(t);
  if (k != 1 || n != ((rows + 127) / 128) * ((cols + 127) / 128)) {
    PyErr_Format(PyExc_ValueError, "%s must hold one fp32 scale per 128 x 128 tile of %lld x %lld", name,
                 (long long)rows, (long long)cols);
    return -1;
  }
  return contiguous(x, name) ? -1 : pointer_of(dev, x, name, p);
}

/* a contiguous tensor of any type and shape: its address and bytes */
static int workspace(int64_t* dev, PyObject* x, int64_t* p, int64_t* bytes) {
  if (x == Py_None) {
    PyErr_SetString(PyExc_ValueError, "ws is None");
    return -1;
  }
  if (contiguous(x, "ws")) return -1;
  PyObject* v = PyObject_GetAttr(x, s_nbytes);
  if (!v) return -1;
  *bytes = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : pointer_of(dev, x, "ws", p);
}

/* the library launches on the current device: it must be the tensors' */
static int on_current(int64_t dev) {
  PyObject* v = PyObject_CallNoArgs(g_current);
  if (!v) return 0;
  const int64_t d = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (d != dev && !PyErr_Occurred())
    PyErr_Format(PyExc_ValueError, "the tensors are on GPU %lld, the current device is %lld", (long long)dev, (long long)d);
  return !PyErr_Occurred();
}

/* FP8 rows: codes and their scales [ceil(cols / 128), n] */
static int code_rows(int64_t* dev, PyObject* codes, PyObject* scale, int64_t n, int64_t cols, Mat* c, Mat* s) {
  if (mat(dev, codes, "codes", FP8, n, cols, c)) return -1;
  return mat(dev, scale, "code_scale", FP32, (c->cols + 127) / 128, c->rows, s);
}

/* the start of every call */
static int args_are(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, want);
  return n == want;
}

static int64_t word(double v) {
  int64_t w;
  memcpy(&w, &v, 8);
  return w;
}

static int integer(PyObject* o, int64_t* v) {
  *v = (int64_t)PyLong_AsUnsignedLongLongMask(o);
  return PyErr_Occurred() ? -1 : 0;
}

#define RUN(op, ...)                             \
  do {                                           \
    const int64_t words_[] = {__VA_ARGS__};      \
    int rc;                                      \
    if (!on_current(dev)) return NULL;           \
    Py_BEGIN_ALLOW_THREADS rc = g_call(op, words_);  \
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc); \
  } while (0)

/* a stream comes as an integer */

static PyObject* f_embed(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* table ids out scale table_scale stream */
  int64_t dev = -1;
  Mat t, o;
  int64_t ids, bits, count, ts = 0, st;
  if (!args_are(n, 6) || mat(&dev, a[0], "table", BF16 | FP8, -1, -1, &t) || vec(&dev, a[1], "ids", 0, -1, &ids, &bits, &count) ||
      mat(&dev, a[2], "out", BF16, count, t.cols, &o) || (t.kind == 2 && tiles(&dev, a[4], "table_scale", t.rows, t.cols, &ts)) ||
      integer(a[5], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) return NULL;
  RUN(0, t.p, t.kind, ts, t.rows, t.cols, t.ld, ids, bits, count, word(f), o.p, o.ld, st);
}

static PyObject* f_embed_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* dy ids out ws scale accumulate stream */
  int64_t dev = -1;
  Mat d, o;
  int64_t ids, bits, count, ws, wb, st;
  if (!args_are(n, 7) || vec(&dev, a[1], "ids", 0, -1, &ids, &bits, &count) || mat(&dev, a[2], "out", BF16 | FP32, -1, -1, &o) ||
      mat(&dev, a[0], "dy", BF16, count, o.cols, &d) || workspace(&dev, a[3], &ws, &wb) || integer(a[6], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[4]);
  const int acc = PyObject_IsTrue(a[5]);
  if (PyErr_Occurred()) return NULL;
  RUN(1, d.p, d.ld, ids, bits, count, word(f), o.rows, o.cols, o.p, o.kind, o.ld, acc, ws, wb, st);
}

static PyObject* f_rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* x weight eps residual h y codes code_scale rstd stream */
  int64_t dev = -1;
  Mat x, r, h, y, c, s;
  int64_t w, q = 0, st;
  if (!args_are(n, 10) || mat(&dev, a[0], "x", BF16, -1, -1, &x) || vec(&dev, a[1], "weight", BF16, x.cols, &w, NULL, NULL) ||
      opt(&dev, a[3], "residual", BF16, x.rows, x.cols, &r) || opt(&dev, a[4], "h", BF16, x.rows, x.cols, &h) ||
      opt(&dev, a[5], "y", BF16, x.rows, x.cols, &y))
    return NULL;
  memset(&c, 0, sizeof c);
  memset(&s, 0, sizeof s);
  if (a[6] != Py_None && code_rows(&dev, a[6], a[7], x.rows, x.cols, &c, &s)) return NULL;
  if ((a[8] != Py_None && vec(&dev, a[8], "rstd", FP32, x.rows, &q, NULL, NULL)) || integer(a[9], &st)) return NULL;
  const double eps = PyFloat_AsDouble(a[2]);
  if (PyErr_Occurred()) return NULL;
  RUN(2, x.p, x.ld, r.p, r.ld, w, word(eps), x.rows, x.cols, h.p, h.ld, y.p, y.ld, c.p, c.ld, s.p, s.ld, q, st);
}

static PyObject* f_rmsnorm_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* dy h weight rstd dx dw ws dh accumulate stream */
  int64_t dev = -1;
  Mat y, h, g, x;
  int64_t w, q, dw, kind, ws, wb, st;
  if (!args_are(n, 10) || mat(&dev, a[1], "h", BF16, -1, -1, &h) || mat(&dev, a[0], "dy", BF16, h.rows, h.cols, &y) ||
      vec(&dev, a[2], "weight", BF16, h.cols, &w, NULL, NULL) || vec(&dev, a[3], "rstd", FP32, h.rows, &q, NULL, NULL) ||
      mat(&dev, a[4], "dx", BF16, h.rows, h.cols, &x) || vec(&dev, a[5], "dw", BF16 | FP32, h.cols, &dw, &kind, NULL) ||
      opt(&dev, a[7], "dh", BF16, h.rows, h.cols, &g) || workspace(&dev, a[6], &ws, &wb) || integer(a[9], &st))
    return NULL;
  const int acc = PyObject_IsTrue(a[8]);
  if (PyErr_Occurred()) return NULL;
  RUN(3, y.p, y.ld, h.p, h.ld, w, q, g.p, g.ld, h.rows, h.cols, x.p, x.ld, dw, kind, acc, ws, wb, st);
}

static PyObject* f_quant_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* x codes code_scale stream */
  int64_t dev = -1;
  Mat x, c, s;
  int64_t st;
  if (!args_are(n, 4) || mat(&dev, a[0], "x", BF16, -1, -1, &x) || code_rows(&dev, a[1], a[2], x.rows, x.cols, &c, &s) ||
      integer(a[3], &st))
    return NULL;
  RUN(4, x.p, x.ld, x.rows, x.cols, c.p, c.ld, s.p, s.ld, st);
}

static PyObject* f_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* codes code_scale w w_scale out ws stream */
  int64_t dev = -1;
  Mat c, s, w, o;
  int64_t ts, ws, wb, st;
  if (!args_are(n, 7) || mat(&dev, a[2], "w", FP8, -1, -1, &w) || code_rows(&dev, a[0], a[1], -1, w.cols, &c, &s) ||
      tiles(&dev, a[3], "w_scale", w.rows, w.cols, &ts) || mat(&dev, a[4], "out", BF16, c.rows, w.rows, &o) ||
      workspace(&dev, a[5], &ws, &wb) || integer(a[6], &st))
    return NULL;
  RUN(5, c.p, c.ld, s.p, s.ld, w.p, w.ld, ts, c.rows, w.rows, w.cols, o.p, o.ld, ws, wb, st);
}

static PyObject* f_linear_dx(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* dy w w_scale dx ws stream */
  int64_t dev = -1;
  Mat y, w, x;
  int64_t ts, ws, wb, st;
  if (!args_are(n, 6) || mat(&dev, a[1], "w", FP8, -1, -1, &w) || mat(&dev, a[0], "dy", BF16, -1, w.rows, &y) ||
      tiles(&dev, a[2], "w_scale", w.rows, w.cols, &ts) || mat(&dev, a[3], "dx", BF16, y.rows, w.cols, &x) ||
      workspace(&dev, a[4], &ws, &wb) || integer(a[5], &st))
    return NULL;
  RUN(6, y.p, y.ld, w.p, w.ld, ts, y.rows, w.rows, w.cols, x.p, x.ld, ws, wb, st);
}

static PyObject* f_linear_dw(PyObject* self, PyObject* const* a, Py_ssize_t n) { /* dy codes code_scale dw ws accumulate stream */
  int64_t dev = -1;
  Mat y, c, s, d;
  int64_t ws, wb, st;
  if (!args_are(n, 7) || mat(&dev, a[0], "dy", BF16, -1, -1, &y) || code_rows(&dev, a[1], a[2], y.rows, -1, &c, &s) ||
      mat(&dev, a[3], "dw", BF16, y.cols, c.cols, &d) || workspace(&dev, a[4], &ws, &wb) || integer(a[6], &st))
    return NULL;
  const int acc = PyObject_IsTrue(a[5]);
  if (PyErr_Occurred()) return NULL;
  RUN(7, y.p, y.ld, c.p, c.ld, s.p, s.ld, c.rows, y.cols, c.cols, d.p, d.ld, acc, ws, wb, st);
}

/* the rows and the weight of a loss: a[0 .. 3] codes code_scale w w_scale */
static int loss_head(int64_t* dev, PyObject* const* a, Mat* c, Mat* s, Mat* w, int64_t* ts) {
  return mat(dev, a[2], "w", FP8, -1, -1, w) || code_rows(dev, a[0], a[1], -1, w->cols, c, s) ||
         tiles(dev, a[3], "w_scale", w->rows, w->cols, ts);
}

static PyObject* f_cross_entropy(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* codes code_scale w w_scale targets loss lse ws scale stream */
  int64_t dev = -1;
  Mat c, s, w;
  int64_t ts, y, bits, loss, lse, ws, wb, st;
  if (!args_are(n, 10) || loss_head(&dev, a, &c, &s, &w, &ts) || vec(&dev, a[4], "targets", 0, c.rows, &y, &bits, NULL) ||
      vec(&dev, a[5], "loss", FP32, c.rows, &loss, NULL, NULL) || vec(&dev, a[6], "lse", FP32, c.rows, &lse, NULL, NULL) ||
      workspace(&dev, a[7], &ws, &wb) || integer(a[9], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return NULL;
  RUN(8, c.p, c.ld, s.p, s.ld, w.p, w.ld, ts, c.rows, w.rows, w.cols, y, bits, word(f), loss, lse, ws, wb, st);
}

static PyObject* f_cross_entropy_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* codes code_scale w w_scale targets loss lse dloss dx dw ws scale accumulate stream */
  int64_t dev = -1;
  Mat c, s, w, dx, dw;
  int64_t ts, y, bits, loss, lse, dl, ws, wb, st;
  if (!args_are(n, 14) || loss_head(&dev, a, &c, &s, &w, &ts) || vec(&dev, a[4], "targets", 0, c.rows, &y, &bits, NULL) ||
      vec(&dev, a[5], "loss", FP32, c.rows, &loss, NULL, NULL) || vec(&dev, a[6], "lse", FP32, c.rows, &lse, NULL, NULL) ||
      vec(&dev, a[7], "dloss", FP32, c.rows, &dl, NULL, NULL) || opt(&dev, a[8], "dx", BF16, c.rows, w.cols, &dx) ||
      opt(&dev, a[9], "dw", BF16, w.rows, w.cols, &dw) || workspace(&dev, a[10], &ws, &wb) || integer(a[13], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[11]);
  const int acc = PyObject_IsTrue(a[12]);
  if (PyErr_Occurred()) return NULL;
  RUN(9, c.p, c.ld, s.p, s.ld, w.p, w.ld, ts, c.rows, w.rows, w.cols, y, bits, word(f), loss, lse, dl, dx.p, dx.ld, dw.p,
      dw.ld, acc, ws, wb, st);
}

static PyObject* f_distill(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* codes code_scale w w_scale ids teacher loss lse logp ws scale stream */
  int64_t dev = -1;
  Mat c, s, w, y, z, p;
  int64_t ts, loss, lse, ws, wb, st;
  if (!args_are(n, 12) || loss_head(&dev, a, &c, &s, &w, &ts) || id_mat(&dev, a[4], "ids", c.rows, -1, &y) ||
      mat(&dev, a[5], "teacher", BF16 | FP32, c.rows, y.cols, &z) || vec(&dev, a[6], "loss", FP32, c.rows, &loss, NULL, NULL) ||
      vec(&dev, a[7], "lse", FP32, c.rows, &lse, NULL, NULL) || mat(&dev, a[8], "logp", FP32, c.rows, y.cols, &p) ||
      workspace(&dev, a[9], &ws, &wb) || integer(a[11], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  RUN(10, c.p, c.ld, s.p, s.ld, w.p, w.ld, ts, c.rows, w.rows, w.cols, y.p, y.kind, y.ld, z.p, z.kind, z.ld, y.cols, word(f),
      loss, lse, p.p, p.ld, ws, wb, st);
}

static PyObject* f_distill_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  /* codes code_scale w w_scale ids teacher lse logp dloss dx dw ws scale accumulate stream */
  int64_t dev = -1;
  Mat c, s, w, y, z, p, dx, dw;
  int64_t ts, lse, dl, ws, wb, st;
  if (!args_are(n, 15) || loss_head(&dev, a, &c, &s, &w, &ts) || id_mat(&dev, a[4], "ids", c.rows, -1, &y) ||
      mat(&dev, a[5], "teacher", BF16 | FP32, c.rows, y.cols, &z) || vec(&dev, a[6], "lse", FP32, c.rows, &lse, NULL, NULL) ||
      mat(&dev, a[7], "logp", FP32, c.rows, y.cols, &p) || vec(&dev, a[8], "dloss", FP32, c.rows, &dl, NULL, NULL) ||
      opt(&dev, a[9], "dx", BF16, c.rows, w.cols, &dx) || opt(&dev, a[10], "dw", BF16, w.rows, w.cols, &dw) ||
      workspace(&dev, a[11], &ws, &wb) || integer(a[14], &st))
    return NULL;
  const double f = PyFloat_AsDouble(a[12]);
  const int acc = PyObject_IsTrue(a[13]);
  if (PyErr_Occurred()) return NULL;
  RUN(11, c.p, c.ld, s.p, s.ld, w.p, w.ld, ts, c.rows, w.rows, w.cols, y.p, y.kind, y.ld, z.p, z.kind, z.ld, y.cols, word(f),
      lse, p.p, p.ld, dl, dx.p, dx.ld, dw.p, dw.ld, acc, ws, wb, st);
}

/* the workspace of a check: (address, bytes) */
static PyObject* f_workspace(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  int64_t dev = -1, p, bytes;
  if (!args_are(n, 1) || workspace(&dev, a[0], &p, &bytes) || !on_current(dev)) return NULL;
  return Py_BuildValue("LL", (long long)p, (long long)bytes);
}

/* bind(address of bq_call, dict of kinds, function that adds to it, current device's function) */
static PyObject* f_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!args_are(n, 4)) return NULL;
  void* p = PyLong_AsVoidPtr(a[0]);
  if (PyErr_Occurred()) return NULL;
  if (!PyDict_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "kinds must be a dict");
    return NULL;
  }
  memcpy(&g_call, &p, sizeof p);
  Py_INCREF(a[1]);
  Py_XSETREF(g_kinds, a[1]);
  Py_INCREF(a[2]);
  Py_XSETREF(g_fill, a[2]);
  Py_INCREF(a[3]);
  Py_XSETREF(g_current, a[3]);
  Py_RETURN_NONE;
}

#define FN(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    FN("bind", f_bind),
    FN("embed", f_embed),
    FN("embed_grad", f_embed_grad),
    FN("rmsnorm", f_rmsnorm),
    FN("rmsnorm_grad", f_rmsnorm_grad),
    FN("quant_rows_fp8", f_quant_rows),
    FN("linear_fp8", f_linear),
    FN("linear_fp8_dx", f_linear_dx),
    FN("linear_fp8_dw", f_linear_dw),
    FN("cross_entropy_fp8", f_cross_entropy),
    FN("cross_entropy_fp8_grad", f_cross_entropy_grad),
    FN("distill_fp8", f_distill),
    FN("distill_fp8_grad", f_distill_grad),
    FN("workspace", f_workspace),
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bqcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__bqcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_is_contiguous || !s_get_device || !s_nbytes) return NULL;
  return PyModule_Create(&module);
}
