/* binding.c - CPython fast path of the operators around the layer.
 *
 * Reads what moe_linear, moe_route and moe_rmsnorm_quantize need of their
 * tensors (type, shape, strides, device, address) through the C API and makes
 * the call: a small operator takes a few microseconds on the GPU, and the same
 * reads in Python with a ctypes call of twenty arguments took four on the host
 * (7.4 us a call in all, 4.1 with this).
 *
 * Only well-formed calls are made here: two-dimensional operands with dense
 * rows, dense vectors of the expected type and length, everything on the current
 * device. For anything else a function returns None, and its caller in capi.py
 * repeats the checks there, which name the fault. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef int (*linear_fn)(int, const void*, int64_t, const float*, const void*, int64_t, const float*, int, const void*,
                         int, int, const void*, int64_t, void*, int, int64_t, int, int, int, void*);
typedef int (*route_fn)(const void*, int, int64_t, const float*, const uint8_t*, const int32_t*, int, int, int, int,
                        int, int, int, int, float, int32_t*, float*, void*);
typedef int (*norm_fn)(int, int, const void*, const void*, const void*, int, float, int, int, void*, void*, void*,
                       void*, void*);

static linear_fn f_linear;
static route_fn f_route;
static norm_fn f_norm;

/* dtype codes of include/moe_b200.h, and two more for bytes */
enum { BF16 = 0, FP16 = 1, E4M3 = 2, F32 = 4, U8 = 16, BOOL = 17, I32 = 18, N_TYPES = 7 };
static const int type_code[N_TYPES] = {BF16, FP16, F32, E4M3, U8, BOOL, I32};
static PyObject* type_obj[N_TYPES];
static PyObject *get_device_fn, *get_stream_fn;
static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_data_ptr, *s_numel, *s_is_contiguous, *s_cuda_stream;

typedef struct {
  void* ptr;
  long long rows, cols, ld; /* operands; a vector has rows = elements */
  int type;
} tensor_t;

static int long_of(PyObject* o, long long* v) { /* steals o */
  if (!o) return 0;
  *v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  const int ok = PyLong_Check(o) && !(*v == -1 && PyErr_Occurred());
  Py_DECREF(o);
  return ok;
}

static int pair_of(PyObject* o, long long* a, long long* b) { /* steals o */
  if (!o) return 0;
  int ok = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2;
  if (ok) {
    *a = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0));
    *b = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1));
    ok = !PyErr_Occurred();
  }
  Py_DECREF(o);
  return ok;
}

/* type, device (must be `dev`) and address of a tensor */
static int common(PyObject* t, long long dev, tensor_t* o) {
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  o->type = -1;
  for (int i = 0; i < N_TYPES; ++i)
    if (d == type_obj[i]) o->type = type_code[i];
  Py_DECREF(d);
  long long v;
  if (o->type < 0 || !long_of(PyObject_CallMethodNoArgs(t, s_get_device), &v) || v != dev) return 0;
  PyObject* p = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!p) return 0;
  o->ptr = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

/* a [rows, cols] operand with dense rows */
static int operand(PyObject* t, long long dev, tensor_t* o) {
  long long step;
  if (!common(t, dev, o) || !pair_of(PyObject_GetAttr(t, s_shape), &o->rows, &o->cols) ||
      !pair_of(PyObject_CallMethodNoArgs(t, s_stride), &o->ld, &step))
    return 0;
  if ((step != 1 && o->cols != 1) || o->rows < 1 || o->rows > INT32_MAX || o->cols > INT32_MAX) return 0;
  if (o->rows == 1) o->ld = (o->cols + 15) / 16 * 16; /* the stride of a single row says nothing */
  return o->ld >= o->cols;
}

/* a dense tensor of any shape with elements; None: a null pointer (which an empty
 * tensor's address would be too) */
static int vector(PyObject* t, long long dev, tensor_t* o) {
  o->ptr = NULL;
  o->rows = 0;
  o->type = -1;
  if (t == Py_None) return 1;
  if (!common(t, dev, o) || !long_of(PyObject_CallMethodNoArgs(t, s_numel), &o->rows) || o->rows < 1) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
  const int ok = c == Py_True;
  Py_XDECREF(c);
  return ok;
}

static int current(PyObject* stream, long long* dev, void** s) {
  if (!long_of(PyObject_CallNoArgs(get_device_fn), dev) || *dev < 0) return 0;
  PyObject* h;
  if (stream == Py_None) {
    PyObject* d = PyLong_FromLongLong(*dev);
    h = d ? PyObject_CallOneArg(get_stream_fn, d) : NULL;
    Py_XDECREF(d);
  } else {
    h = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (!h) return 0;
  *s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

static PyObject* not_plain(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

static int int_of(PyObject* o, int* v) {
  const long l = PyLong_AsLong(o);
  *v = (int)l;
  return !PyErr_Occurred() && l == *v;
}

static int is_float(int type) { return type == BF16 || type == FP16 || type == F32; }

/* linear(dtype, x, x_scale, w, w_scale, bias, act, residual, out, stream) */
static PyObject* py_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 10 || !f_linear) return not_plain();
  int dtype, act;
  long long dev;
  void* s;
  tensor_t x, xs, w, ws, b, r, o;
  if (!int_of(a[0], &dtype) || !int_of(a[6], &act) || !current(a[9], &dev, &s) || !operand(a[1], dev, &x) ||
      !operand(a[3], dev, &w) || !operand(a[8], dev, &o) || !vector(a[2], dev, &xs) || !vector(a[4], dev, &ws) ||
      !vector(a[5], dev, &b))
    return not_plain();
  r.ptr = NULL;
  r.ld = 0;
  if (a[7] != Py_None &&
      (!operand(a[7], dev, &r) || r.type != o.type || r.rows != o.rows || r.cols != o.cols))
    return not_plain();
  const int want = dtype == E4M3 ? (x.type == U8 ? U8 : E4M3) : dtype;
  const int w_ok = dtype == E4M3 ? (w.type == U8 || w.type == E4M3) : w.type == dtype;
  if ((dtype != BF16 && dtype != FP16 && dtype != E4M3) || x.type != want || !w_ok || !is_float(o.type) ||
      w.cols != x.cols || o.rows != x.rows || o.cols != w.rows || (xs.ptr && (xs.type != F32 || xs.rows != x.rows)) ||
      (ws.ptr && (ws.type != F32 || ws.rows > INT32_MAX)) || (b.ptr && (!is_float(b.type) || b.rows != w.rows)))
    return not_plain();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_linear(dtype, x.ptr, x.ld, xs.ptr, w.ptr, w.ld, ws.ptr, ws.ptr ? (int)ws.rows : 1, b.ptr,
                    b.ptr ? b.type : F32, act, r.ptr, r.ld, o.ptr, o.type, o.ld, (int)x.rows, (int)w.rows,
                    (int)x.cols, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

/* route(logits, bias, expert_mask, num_valid, top_k, score, n_group, topk_group, group_score, renormalize, rsf,
 *       topk_ids, topk_weights, stream) */
static PyObject* py_route(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 14 || !f_route) return not_plain();
  int k, score, n_group, topk_group, group_score;
  long long dev;
  void* s;
  tensor_t l, b, m, nv, ids, w;
  const int renorm = PyObject_IsTrue(a[9]);
  const double rsf = PyFloat_AsDouble(a[10]);
  if (renorm < 0 || PyErr_Occurred() || !int_of(a[4], &k) || !int_of(a[5], &score) || !int_of(a[6], &n_group) ||
      !int_of(a[7], &topk_group) || !int_of(a[8], &group_score) || !current(a[13], &dev, &s) ||
      !operand(a[0], dev, &l) || !vector(a[1], dev, &b) || !vector(a[2], dev, &m) || !vector(a[3], dev, &nv) ||
      !vector(a[11], dev, &ids) || !vector(a[12], dev, &w))
    return not_plain();
  const long long slots = l.rows * k;
  if (!is_float(l.type) || (b.ptr && (b.type != F32 || b.rows != l.cols)) ||
      (m.ptr && ((m.type != U8 && m.type != BOOL) || m.rows != l.cols)) ||
      (nv.ptr && (nv.type != I32 || nv.rows != 1)) || ids.type != I32 || ids.rows != slots || w.type != F32 ||
      w.rows != slots)
    return not_plain();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_route(l.ptr, l.type, l.ld, b.ptr, m.ptr, nv.ptr, (int)l.rows, (int)l.cols, k, score, n_group, topk_group,
                   group_score, renorm, (float)rsf, ids.ptr, w.ptr, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

/* rmsnorm_quantize(quant, x, residual, gamma, eps, residual_out, y, codes, scale, stream); quant -1: none */
static PyObject* py_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (n != 10 || !f_norm) return not_plain();
  int quant;
  long long dev;
  void* s;
  tensor_t x, r, g, ro, y, c, sc;
  const double eps = PyFloat_AsDouble(a[4]);
  if (PyErr_Occurred() || !int_of(a[0], &quant) || !current(a[9], &dev, &s) || !operand(a[1], dev, &x) ||
      !vector(a[2], dev, &r) || !vector(a[3], dev, &g) || !vector(a[5], dev, &ro) || !vector(a[6], dev, &y) ||
      !vector(a[7], dev, &c) || !vector(a[8], dev, &sc))
    return not_plain();
  const long long all = x.rows * x.cols;
  const int mx = quant == 3;
  if ((x.type != BF16 && x.type != FP16) || (x.rows > 1 && x.ld != x.cols) ||
      (r.ptr && (r.type != x.type || r.rows != all)) || (g.type != x.type && g.type != F32) || g.rows != x.cols ||
      (ro.ptr && (ro.type != x.type || ro.rows != all)) || (y.ptr && (y.type != x.type || y.rows != all)) ||
      (c.ptr && ((c.type != U8 && c.type != E4M3) || c.rows != all)) ||
      (sc.ptr && (sc.type != (mx ? U8 : F32) || sc.rows != (mx ? all / 32 : x.rows))))
    return not_plain();
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f_norm(x.type, quant, x.ptr, r.ptr, g.ptr, g.type, (float)eps, (int)x.rows, (int)x.cols, ro.ptr, y.ptr,
                  c.ptr, sc.ptr, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

/* init((linear, route, rmsnorm addresses), (bf16, fp16, f32, e4m3, uint8, bool, int32), current_device, current_stream) */
static PyObject* py_init(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *fns, *types, *dev, *stream;
  if (!PyArg_ParseTuple(args, "O!O!OO", &PyTuple_Type, &fns, &PyTuple_Type, &types, &dev, &stream)) return NULL;
  if (PyTuple_GET_SIZE(fns) != 3 || PyTuple_GET_SIZE(types) != N_TYPES) {
    PyErr_SetString(PyExc_ValueError, "three functions and seven types");
    return NULL;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(fns, i));
  if (PyErr_Occurred()) return NULL;
  for (int i = 0; i < N_TYPES; ++i) {
    Py_INCREF(PyTuple_GET_ITEM(types, i));
    Py_XSETREF(type_obj[i], PyTuple_GET_ITEM(types, i));
  }
  Py_INCREF(dev);
  Py_XSETREF(get_device_fn, dev);
  Py_INCREF(stream);
  Py_XSETREF(get_stream_fn, stream);
  f_linear = (linear_fn)p[0];
  f_route = (route_fn)p[1];
  f_norm = (norm_fn)p[2];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", py_init, METH_VARARGS, "Entry points, types and the current device's functions."},
    {"linear", (PyCFunction)(void (*)(void))py_linear, METH_FASTCALL, "moe_linear: a status, or None."},
    {"route", (PyCFunction)(void (*)(void))py_route, METH_FASTCALL, "moe_route: a status, or None."},
    {"rmsnorm_quantize", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL, "moe_rmsnorm_quantize: a status, or None."},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_numel = PyUnicode_InternFromString("numel");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
