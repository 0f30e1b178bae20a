/* marshal.c -- argument marshalling of the checked entry points (RMSNorm, MXFP4,
 * three-axis RoPE) for the Python binding, as a CPython extension module.
 *
 * The C ABI takes bare pointers, so these calls check every tensor they are given:
 * element type, device, contiguity and shape.  In Python, with ctypes for the call,
 * that is most of a small call's time (RMSNorm of one row: 3 of 6 us, the launch
 * itself 2).  Here the same attributes are asked for from C and the entry point is
 * called directly.  The module knows tensors by their methods only (dtype, shape,
 * get_device, is_contiguous, stride, numel, data_ptr): it is built without torch's
 * headers, and computes nothing.
 *
 * Each method returns the entry point's vit_status, or VIT_ERR_INVALID_ARG for a
 * tensor of another type, device or layout and VIT_ERR_SHAPE for one of another
 * shape or too few bytes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "../../include/vit.h"

/* The entry points, by address (bind()): the library is loaded by the package. */
static struct {
  __typeof__(&vit_rmsnorm) rmsnorm;
  __typeof__(&vit_rmsnorm_mx8) rmsnorm_mx8;
  __typeof__(&vit_mx4_quantize) mx4_quantize;
  __typeof__(&vit_mx4_dequantize) mx4_dequantize;
  __typeof__(&vit_linear_mx4) linear_mx4;
  __typeof__(&vit_rope3d) rope3d;
} lib;

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_numel,
    *s_stride, *s_cuda_stream;

/* One context's calls: its handle, device and element type. */
typedef struct {
  PyObject_HEAD
  vit_ctx *ctx;
  PyObject *element, *u8, *i32, *current; /* dtypes; device -> current raw stream */
  long device, head_dim;
  float eps;
} Calls;

enum { kRaised = -1 }; /* a Python exception is set */

/* A method's integer result. */
static int ask(PyObject *t, PyObject *name, unsigned long long *v) {
  PyObject *r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return kRaised;
  *v = PyLong_AsUnsignedLongLongMask(r);
  Py_DECREF(r);
  return PyErr_Occurred() ? kRaised : VIT_OK;
}

/* Type and device of a tensor, and its address. */
static int check_place(const Calls *c, PyObject *t, PyObject *dtype, void **p) {
  unsigned long long v;
  PyObject *a = PyObject_GetAttr(t, s_dtype);
  if (!a) return kRaised;
  Py_DECREF(a);
  if (a != dtype) return VIT_ERR_INVALID_ARG; /* dtypes are singletons */
  if (ask(t, s_get_device, &v)) return kRaised;
  if ((long)v != c->device) return VIT_ERR_INVALID_ARG;
  if (ask(t, s_data_ptr, &v)) return kRaised;
  *p = (void *)(uintptr_t)v;
  return VIT_OK;
}

static int check_contiguous(PyObject *t) {
  PyObject *a = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  if (!a) return kRaised;
  const int yes = a == Py_True;
  Py_DECREF(a);
  return yes ? VIT_OK : VIT_ERR_INVALID_ARG;
}

/* The n sizes of a tensor with n dimensions. */
static int get_sizes(PyObject *t, PyObject *name, int method, Py_ssize_t n, long long *v) {
  PyObject *a = method ? PyObject_CallMethodNoArgs(t, name) : PyObject_GetAttr(t, name);
  if (!a) return kRaised;
  int s = PyTuple_Check(a) && PyTuple_GET_SIZE(a) == n ? VIT_OK : VIT_ERR_SHAPE;
  for (Py_ssize_t i = 0; s == VIT_OK && i < n; ++i) {
    v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a, i));
    if (v[i] == -1 && PyErr_Occurred()) s = kRaised;
  }
  Py_DECREF(a);
  return s;
}

/* A contiguous tensor of this type and shape (n sizes), or None where it may be. */
static int check_dense(const Calls *c, PyObject *t, PyObject *dtype, Py_ssize_t n,
                       const long long *shape, int optional, void **p) {
  long long got[3];
  int s;
  *p = NULL;
  if (optional && t == Py_None) return VIT_OK;
  if ((s = check_place(c, t, dtype, p)) || (s = check_contiguous(t)) ||
      (s = get_sizes(t, s_shape, 0, n, got)))
    return s;
  for (Py_ssize_t i = 0; i < n; ++i)
    if (got[i] != shape[i]) return VIT_ERR_SHAPE;
  return VIT_OK;
}

/* Codes and scales of a [rows, K] matrix: byte tensors of at least its sizes. */
static int check_codes(const Calls *c, PyObject *codes, PyObject *scales, long long rows,
                       long long row_bytes, long long K, void **pc, void **ps) {
  unsigned long long nc, ns;
  int s;
  if ((s = check_place(c, codes, c->u8, pc)) || (s = check_contiguous(codes)) ||
      (s = check_place(c, scales, c->u8, ps)) || (s = check_contiguous(scales)) ||
      (s = ask(codes, s_numel, &nc)) || (s = ask(scales, s_numel, &ns)))
    return s;
  return nc < (unsigned long long)(rows * row_bytes) ||
                 ns < (unsigned long long)((rows + 127) / 128 * ((K + 127) / 128) * 512)
             ? VIT_ERR_SHAPE
             : VIT_OK;
}

/* Sizes that the C ABI's int takes. */
static int fits_int(const long long *v, int n) {
  for (int i = 0; i < n; ++i)
    if (v[i] > INT_MAX) return VIT_ERR_UNSUPPORTED;
  return VIT_OK;
}

/* A choice (an enum of the C ABI) that its int holds. */
static int is_int(long v) { return v >= INT_MIN && v <= INT_MAX; }

/* The given stream (an integer, or an object with cuda_stream), or the device's
 * current one. */
static int get_stream(const Calls *c, PyObject *o, void **st) {
  PyObject *v;
  if (o == Py_None) {
    PyObject *dev = PyLong_FromLong(c->device);
    if (!dev) return kRaised;
    v = PyObject_CallOneArg(c->current, dev);
    Py_DECREF(dev);
  } else if (PyLong_Check(o)) {
    v = Py_NewRef(o);
  } else {
    v = PyObject_GetAttr(o, s_cuda_stream);
  }
  if (!v) return kRaised;
  *st = (void *)(uintptr_t)PyLong_AsUnsignedLongLongMask(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? kRaised : VIT_OK;
}

static int get_eps(const Calls *c, PyObject *o, float *eps) {
  *eps = o == Py_None ? c->eps : (float)PyFloat_AsDouble(o);
  return PyErr_Occurred() ? kRaised : VIT_OK;
}

static int arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are wanted", n, want);
  return 0;
}

static PyObject *result(int s) { return s == kRaised ? NULL : PyLong_FromLong(s); }

#define LAUNCH(call)       \
  do {                     \
    Py_BEGIN_ALLOW_THREADS \
    s = (int)(call);       \
    Py_END_ALLOW_THREADS   \
  } while (0)

/* x, gamma, y, residual, h, eps, stream */
static PyObject *calls_rmsnorm(Calls *c, PyObject *const *a, Py_ssize_t n) {
  long long sh[2];
  void *x, *g, *y, *r, *h, *st;
  float eps;
  int s;
  if (!arity(n, 7)) return NULL;
  if ((s = get_sizes(a[0], s_shape, 0, 2, sh)) || (s = fits_int(sh, 2)) ||
      (s = check_dense(c, a[0], c->element, 2, sh, 0, &x)) ||
      (s = check_dense(c, a[1], c->element, 1, sh + 1, 0, &g)) ||
      (s = check_dense(c, a[2], c->element, 2, sh, 0, &y)) ||
      (s = check_dense(c, a[3], c->element, 2, sh, 1, &r)) ||
      (s = check_dense(c, a[4], c->element, 2, sh, 1, &h)) || (s = get_eps(c, a[5], &eps)) ||
      sh[0] == 0 || (s = get_stream(c, a[6], &st)))
    return result(s); /* an empty tensor has no address to pass */
  LAUNCH(lib.rmsnorm(c->ctx, x, r, g, h, y, (int)sh[0], (int)sh[1], eps, st));
  return result(s);
}

/* x, gamma, codes, scales, residual, h, eps, stream */
static PyObject *calls_rmsnorm_mx8(Calls *c, PyObject *const *a, Py_ssize_t n) {
  long long sh[2];
  void *x, *g, *q, *sc, *r, *h, *st;
  float eps;
  int s;
  if (!arity(n, 8)) return NULL;
  if ((s = get_sizes(a[0], s_shape, 0, 2, sh)) || (s = fits_int(sh, 2)) ||
      (s = check_dense(c, a[0], c->element, 2, sh, 0, &x)) ||
      (s = check_dense(c, a[1], c->element, 1, sh + 1, 0, &g)) ||
      (s = check_codes(c, a[2], a[3], sh[0], (sh[1] + 15) / 16 * 16, sh[1], &q, &sc)) ||
      (s = check_dense(c, a[4], c->element, 2, sh, 1, &r)) ||
      (s = check_dense(c, a[5], c->element, 2, sh, 1, &h)) || (s = get_eps(c, a[6], &eps)) ||
      sh[0] == 0 || (s = get_stream(c, a[7], &st)))
    return result(s);
  LAUNCH(lib.rmsnorm_mx8(c->ctx, x, r, g, h, (int)sh[0], (int)sh[1], eps, q, sc, st));
  return result(s);
}

/* x, codes, scales, stream; to_codes = 0: the other way round */
static PyObject *mx4_convert(Calls *c, PyObject *const *a, Py_ssize_t n, int to_codes) {
  long long sh[2];
  void *x, *q, *sc, *st;
  int s;
  if (!arity(n, 4)) return NULL;
  if ((s = get_sizes(a[0], s_shape, 0, 2, sh)) || (s = fits_int(sh, 2)) ||
      (s = check_dense(c, a[0], c->element, 2, sh, 0, &x)) ||
      (s = check_codes(c, a[1], a[2], sh[0], (sh[1] + 31) / 32 * 16, sh[1], &q, &sc)) ||
      sh[0] == 0 || sh[1] == 0 || (s = get_stream(c, a[3], &st)))
    return result(s);
  if (to_codes)
    LAUNCH(lib.mx4_quantize(c->ctx, x, (int)sh[0], (int)sh[1], q, sc, st));
  else
    LAUNCH(lib.mx4_dequantize(c->ctx, q, sc, (int)sh[0], (int)sh[1], x, st));
  return result(s);
}
static PyObject *calls_mx4_quantize(Calls *c, PyObject *const *a, Py_ssize_t n) {
  return mx4_convert(c, a, n, 1);
}
static PyObject *calls_mx4_dequantize(Calls *c, PyObject *const *a, Py_ssize_t n) {
  return mx4_convert(c, a, n, 0);
}

/* a's codes and scales, w's, bias, residual, y, K, epilogue, stream */
static PyObject *calls_linear_mx4(Calls *c, PyObject *const *a, Py_ssize_t n) {
  long long sh[2], K;
  void *ac, *as, *wc, *ws, *b, *r, *y, *st;
  long epi;
  int s;
  if (!arity(n, 10)) return NULL;
  K = PyLong_AsLongLong(a[7]);
  epi = PyLong_AsLong(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (K < 0 || !is_int(epi)) return result(VIT_ERR_INVALID_ARG);
  const long long row_bytes = (K + 31) / 32 * 16;
  if ((s = get_sizes(a[6], s_shape, 0, 2, sh)) || (s = fits_int(sh, 2)) || (s = fits_int(&K, 1)) ||
      (s = check_dense(c, a[6], c->element, 2, sh, 0, &y)) ||
      (s = check_dense(c, a[5], c->element, 2, sh, 1, &r)) ||
      (s = check_dense(c, a[4], c->element, 1, sh + 1, 1, &b)) ||
      (s = check_codes(c, a[0], a[1], sh[0], row_bytes, K, &ac, &as)) ||
      (s = check_codes(c, a[2], a[3], sh[1], row_bytes, K, &wc, &ws)) || sh[0] == 0 ||
      (s = get_stream(c, a[9], &st)))
    return result(s);
  LAUNCH(lib.linear_mx4(c->ctx, ac, as, wc, ws, b, r, y, (int)sh[0], (int)sh[1], (int)K,
                        (vit_epilogue)epi, st));
  return result(s);
}

/* x [T, heads, d] or y like it: its address and token stride.  Heads lie d apart
 * and elements next to each other; a single token has no stride to go by. */
static int check_heads(const Calls *c, PyObject *t, const long long *sh, void **p,
                       long long *stride) {
  long long got[3], st[3];
  int s;
  if ((s = check_place(c, t, c->element, p)) || (s = get_sizes(t, s_shape, 0, 3, got)) ||
      (s = get_sizes(t, s_stride, 1, 3, st)))
    return s;
  if (got[0] != sh[0] || got[1] != sh[1] || got[2] != sh[2] || sh[2] != c->head_dim)
    return VIT_ERR_SHAPE;
  if (sh[0] && sh[1] && ((sh[1] > 1 && st[1] != sh[2]) || st[2] != 1)) return VIT_ERR_INVALID_ARG;
  *stride = sh[0] <= 1 && st[0] < sh[1] * sh[2] ? sh[1] * sh[2] : st[0];
  return VIT_OK;
}

/* x, pos, sections, layout, out, stream */
static PyObject *calls_rope3d(Calls *c, PyObject *const *a, Py_ssize_t n) {
  long long sh[3], xs, ys, sec[3], psh[2];
  int32_t sections[3];
  void *x, *y, *pos, *st;
  long layout;
  int s;
  if (!arity(n, 6)) return NULL;
  layout = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return NULL;
  if (!is_int(layout)) return result(VIT_ERR_INVALID_ARG);
  PyObject *seq = PySequence_Tuple(a[2]);
  if (!seq) return NULL;
  s = PyTuple_GET_SIZE(seq) == 3 ? VIT_OK : VIT_ERR_SHAPE;
  for (int i = 0; i < 3 && s == VIT_OK; ++i) {
    sec[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
    if (sec[i] == -1 && PyErr_Occurred()) s = kRaised;
    else if (sec[i] < 0 || sec[i] > INT_MAX) s = VIT_ERR_INVALID_ARG;
    else sections[i] = (int32_t)sec[i];
  }
  Py_DECREF(seq);
  if (s || (s = get_sizes(a[0], s_shape, 0, 3, sh)) || (s = fits_int(sh, 3)) ||
      (s = check_heads(c, a[0], sh, &x, &xs)))
    return result(s);
  y = x;
  ys = xs;
  psh[0] = sh[0];
  psh[1] = 3;
  if ((a[4] != Py_None && (s = check_heads(c, a[4], sh, &y, &ys))) ||
      (s = check_dense(c, a[1], c->i32, 2, psh, 0, &pos)) || sh[0] == 0 ||
      (s = get_stream(c, a[5], &st)))
    return result(s);
  LAUNCH(lib.rope3d(c->ctx, x, xs, y, ys, (const int32_t *)pos, (int)sh[0], (int)sh[1], sections,
                    (vit_rope_layout)layout, st));
  return result(s);
}

static PyMethodDef calls_methods[] = {
    {"rmsnorm", (PyCFunction)(void (*)(void))calls_rmsnorm, METH_FASTCALL, NULL},
    {"rmsnorm_mx8", (PyCFunction)(void (*)(void))calls_rmsnorm_mx8, METH_FASTCALL, NULL},
    {"mx4_quantize", (PyCFunction)(void (*)(void))calls_mx4_quantize, METH_FASTCALL, NULL},
    {"mx4_dequantize", (PyCFunction)(void (*)(void))calls_mx4_dequantize, METH_FASTCALL, NULL},
    {"linear_mx4", (PyCFunction)(void (*)(void))calls_linear_mx4, METH_FASTCALL, NULL},
    {"rope3d", (PyCFunction)(void (*)(void))calls_rope3d, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

/* Calls(handle or None, element dtype, uint8, int32, current-stream function,
 * device, eps, head_dim) */
static int calls_init(Calls *c, PyObject *args, PyObject *kw) {
  PyObject *handle, *e, *u8, *i32, *cur;
  long device, head_dim;
  double eps;
  (void)kw;
  if (!PyArg_ParseTuple(args, "OOOOOldl", &handle, &e, &u8, &i32, &cur, &device, &eps, &head_dim))
    return -1;
  c->ctx = handle == Py_None ? NULL : (vit_ctx *)PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return -1;
  Py_XSETREF(c->element, Py_NewRef(e));
  Py_XSETREF(c->u8, Py_NewRef(u8));
  Py_XSETREF(c->i32, Py_NewRef(i32));
  Py_XSETREF(c->current, Py_NewRef(cur));
  c->device = device;
  c->head_dim = head_dim;
  c->eps = (float)eps;
  return 0;
}

static void calls_dealloc(Calls *c) {
  Py_XDECREF(c->element);
  Py_XDECREF(c->u8);
  Py_XDECREF(c->i32);
  Py_XDECREF(c->current);
  Py_TYPE(c)->tp_free((PyObject *)c);
}

static PyTypeObject CallsType = {
    PyVarObject_HEAD_INIT(NULL, 0).tp_name = "_marshal.Calls",
    .tp_basicsize = sizeof(Calls),
    .tp_flags = Py_TPFLAGS_DEFAULT,
    .tp_new = PyType_GenericNew,
    .tp_init = (initproc)calls_init,
    .tp_dealloc = (destructor)calls_dealloc,
    .tp_methods = calls_methods,
};

/* bind(addresses of the six entry points, in the order of `lib`) */
static PyObject *bind(PyObject *self, PyObject *args) {
  unsigned long long p[6];
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5)) return NULL;
  lib.rmsnorm = (__typeof__(lib.rmsnorm))(uintptr_t)p[0];
  lib.rmsnorm_mx8 = (__typeof__(lib.rmsnorm_mx8))(uintptr_t)p[1];
  lib.mx4_quantize = (__typeof__(lib.mx4_quantize))(uintptr_t)p[2];
  lib.mx4_dequantize = (__typeof__(lib.mx4_dequantize))(uintptr_t)p[3];
  lib.linear_mx4 = (__typeof__(lib.linear_mx4))(uintptr_t)p[4];
  lib.rope3d = (__typeof__(lib.rope3d))(uintptr_t)p[5];
  Py_RETURN_NONE;
}

static PyMethodDef module_methods[] = {{"bind", bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, module_methods};

PyMODINIT_FUNC PyInit__marshal(void) {
  struct {
    PyObject **o;
    const char *name;
  } names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},
               {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
               {&s_data_ptr, "data_ptr"}, {&s_numel, "numel"},
               {&s_stride, "stride"},     {&s_cuda_stream, "cuda_stream"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].o = PyUnicode_InternFromString(names[i].name))) return NULL;
  if (PyType_Ready(&CallsType) < 0) return NULL;
  PyObject *m = PyModule_Create(&module);
  if (!m) return NULL;
  if (PyModule_AddObjectRef(m, "Calls", (PyObject *)&CallsType) < 0) {
    Py_DECREF(m);
    return NULL;
  }
  return m;
}
