/*
 * The paged calls' arguments, marshalled in C: what binding.py does for
 * tensors that are as the calls want them, without its time: a decode of one
 * sequence of 701 rows takes 10.8 us instead of 13.7, an append of one token
 * 8.0 instead of 11.7 (the library's launches: 5.5 and 3.7).
 * Anything else than the plain case -- a wrong type, a missing output, a
 * stream of its own -- returns None, and binding.py goes through its own
 * checks and says what is wrong.
 *
 *   setup(Tensor, bfloat16, float32, int32, uint8, device, stream, append,
 *         gather, decode)
 *       the types to compare with, two callables (the current device, and the
 *       handle of a device's current stream), and the addresses of the
 *       library's functions
 *   append(...), gather(...), decode(...)
 *       the status of the call, or None
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <string.h>

#include "moda.h"

static PyObject *g_tensor, *g_bf16, *g_f32, *g_i32, *g_u8, *g_device, *g_stream;
static PyObject *s_dtype, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_shape, *s_stride;
static moda_status (*f_append)(const void*, const void*, const void*, long long, long long, long long,
                               const float*, int, int, int, const int*, const int*, int, int,
                               const moda_paged_kv*, void*, void*, moda_stream_t);
static moda_status (*f_gather)(const moda_paged_kv*, const int*, const int*, int, void*, void*,
                               moda_stream_t);
static moda_status (*f_decode)(const void*, const moda_paged_kv*, const int*, const void*, const void*,
                               long long, long long, long long, int, int, float, void*, float*, float*,
                               size_t, moda_stream_t);

typedef struct {
  void* p;
  long long n[4]; /* shape */
} Ten;

/* A tensor's method without arguments as a whole number; 0 on failure. */
static int ask(PyObject* t, PyObject* name, long long* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) return 0;
  *out = PyLong_AsLongLong(r);
  Py_DECREF(r);
  return !(*out == -1 && PyErr_Occurred());
}

static int numbers(PyObject* tuple, int n, long long* out) {
  if (!tuple || !PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) != n) return 0;
  for (int i = 0; i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] < 0) return 0; /* no shape, and no stride that the calls take */
  }
  return 1;
}

/* t: a tensor of this type and rank on device dev, contiguous if asked for. */
static int ten(PyObject* t, PyObject* dtype, long long dev, int rank, int contiguous, Ten* out) {
  if (!PyObject_TypeCheck(t, (PyTypeObject*)g_tensor)) return 0;
  PyObject* r = PyObject_GetAttr(t, s_dtype);
  if (!r) return 0;
  Py_DECREF(r);
  if (r != dtype) return 0;
  long long at;
  if (!ask(t, s_get_device, &at) || at != dev) return 0;
  if (contiguous) {
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!r) return 0;
    Py_DECREF(r);
    if (r != Py_True) return 0;
  }
  r = PyObject_GetAttr(t, s_shape);
  const int ok = numbers(r, rank, out->n);
  Py_XDECREF(r);
  if (!ok) return 0;
  r = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!r) return 0;
  out->p = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

static int strides(PyObject* t, int rank, long long* out) {
  PyObject* r = PyObject_CallMethodNoArgs(t, s_stride);
  const int ok = numbers(r, rank, out);
  Py_XDECREF(r);
  return ok;
}

static int fits(long long x) { return x >= 0 && x <= INT32_MAX; }

static int current(long long* dev, moda_stream_t* stream) {
  PyObject* d = PyObject_CallNoArgs(g_device);
  if (!d) return 0;
  *dev = PyLong_AsLongLong(d);
  PyObject* s = PyObject_CallOneArg(g_stream, d);
  Py_DECREF(d);
  if (!s) return 0;
  *stream = (moda_stream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

static int cache_of(PyObject* k, PyObject* v, PyObject* table, PyObject* ks, PyObject* vs, long long dev,
                    moda_paged_kv* c) {
  const int mx4 = ks != Py_None || vs != Py_None;
  PyObject* type = mx4 ? g_u8 : g_bf16;
  Ten tk, tv, tt, a, b;
  if (!ten(k, type, dev, 4, 1, &tk) || !ten(v, type, dev, 4, 1, &tv) || !ten(table, g_i32, dev, 2, 1, &tt))
    return 0;
  if (memcmp(tk.n, tv.n, sizeof tk.n) != 0) return 0;
  for (int i = 0; i < 4; ++i)
    if (!fits(tk.n[i])) return 0;
  if (!fits(tt.n[0]) || !fits(tt.n[1]) || tk.n[3] > 4096) return 0;
  memset(c, 0, sizeof *c);
  c->format = mx4 ? MODA_KV_MX4 : MODA_KV_BF16;
  c->num_pages = (int)tk.n[0];
  c->Hk = (int)tk.n[1];
  c->page_size = (int)tk.n[2];
  c->d = (int)tk.n[3] * (mx4 ? 2 : 1);
  c->B = (int)tt.n[0];
  c->max_pages = (int)tt.n[1];
  c->k = tk.p;
  c->v = tv.p;
  c->block_table = (const int*)tt.p;
  if (mx4) {
    if (!ten(ks, g_u8, dev, 4, 1, &a) || !ten(vs, g_u8, dev, 4, 1, &b)) return 0;
    for (int i = 0; i < 3; ++i)
      if (a.n[i] != tk.n[i] || b.n[i] != tk.n[i]) return 0;
    if (a.n[3] != c->d / 32 || b.n[3] != c->d / 32) return 0;
    c->k_scale = a.p;
    c->v_scale = b.p;
  }
  return 1;
}

/* Rows [N, H, d] with dense tokens; their distance. H < 0: any. */
static int rows(PyObject* t, long long dev, long long N, long long H, int d, Ten* out, long long* stride) {
  long long s[3];
  if (!ten(t, g_bf16, dev, 3, 0, out) || !strides(t, 3, s)) return 0;
  if (out->n[0] != N || (H >= 0 && out->n[1] != H) || out->n[2] != d || !fits(out->n[1])) return 0;
  if (s[2] != 1 || (s[1] != d && out->n[1] > 1)) return 0;
  *stride = N > 1 ? s[0] : out->n[1] * d;
  return 1;
}

static PyObject* none(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

/* append(q, k, v, k_pages, v_pages, table, seq, pos, rope, interleaved, k_scales, v_scales, q_out, k_out) */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return none();
  long long dev, qs = 0, ks, vs;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, k, v, seq, pos, rope, qo, ko;
  memset(&q, 0, sizeof q), memset(&rope, 0, sizeof rope), memset(&qo, 0, sizeof qo), memset(&ko, 0, sizeof ko);
  if (!current(&dev, &stream) || !cache_of(a[3], a[4], a[5], a[10], a[11], dev, &c)) return none();
  if (!ten(a[6], g_i32, dev, 1, 1, &seq) || !ten(a[7], g_i32, dev, 1, 1, &pos)) return none();
  const long long N = seq.n[0];
  if (pos.n[0] != N || N < 1 || !fits(N)) return none();
  if (a[0] != Py_None) {
    if (!rows(a[0], dev, N, -1, c.d, &q, &qs)) return none();
    if (!ten(a[12], g_bf16, dev, 3, 1, &qo) || memcmp(qo.n, q.n, 3 * sizeof q.n[0]) != 0) return none();
  } else if (a[12] != Py_None) {
    return none();
  }
  if (!rows(a[1], dev, N, c.Hk, c.d, &k, &ks) || !rows(a[2], dev, N, c.Hk, c.d, &v, &vs)) return none();
  if (a[8] != Py_None && (!ten(a[8], g_f32, dev, 2, 1, &rope) || !fits(rope.n[0]) || !fits(rope.n[1])))
    return none();
  if (a[13] != Py_None &&
      (!ten(a[13], g_bf16, dev, 3, 1, &ko) || memcmp(ko.n, k.n, 3 * sizeof k.n[0]) != 0))
    return none();
  const int inter = PyObject_IsTrue(a[9]);
  if (inter < 0) return none();
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_append(q.p, k.p, v.p, qs, ks, vs, (const float*)rope.p, (int)rope.n[0], (int)rope.n[1], inter,
                (const int*)seq.p, (const int*)pos.p, (int)N, (int)q.n[1], &c, qo.p, ko.p, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* gather(k_pages, v_pages, table, seq, pos, k_scales, v_scales, k, v) */
static PyObject* py_gather(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) return none();
  long long dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten seq, pos, k, v;
  if (!current(&dev, &stream) || !cache_of(a[0], a[1], a[2], a[5], a[6], dev, &c)) return none();
  if (!ten(a[3], g_i32, dev, 1, 1, &seq) || !ten(a[4], g_i32, dev, 1, 1, &pos)) return none();
  const long long N = seq.n[0];
  if (pos.n[0] != N || N < 1 || !fits(N)) return none();
  if (!ten(a[7], g_bf16, dev, 3, 1, &k) || !ten(a[8], g_bf16, dev, 3, 1, &v)) return none();
  if (k.n[0] != N || k.n[1] != c.Hk || k.n[2] != c.d || memcmp(k.n, v.n, 3 * sizeof k.n[0]) != 0)
    return none();
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_gather(&c, (const int*)seq.p, (const int*)pos.p, (int)N, k.p, v.p, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* decode(q, k_pages, v_pages, table, seq_lens, scale, kd, vd, k_scales, v_scales, o, lse, workspace) */
static PyObject* py_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return none();
  long long dev, s1[4] = {0, 0, 0, 1}, s2[4];
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, lens, kd, vd, o, lse, ws;
  memset(&kd, 0, sizeof kd), memset(&vd, 0, sizeof vd), memset(&lse, 0, sizeof lse);
  if (!current(&dev, &stream) || !cache_of(a[1], a[2], a[3], a[8], a[9], dev, &c)) return none();
  if (!ten(a[0], g_bf16, dev, 3, 1, &q) || !ten(a[4], g_i32, dev, 1, 1, &lens)) return none();
  if (c.B < 1 || q.n[0] != c.B || q.n[2] != c.d || !fits(q.n[1]) || lens.n[0] != c.B) return none();
  if (a[6] != Py_None || a[7] != Py_None) {
    if (!ten(a[6], g_bf16, dev, 4, 0, &kd) || !ten(a[7], g_bf16, dev, 4, 0, &vd)) return none();
    if (!strides(a[6], 4, s1) || !strides(a[7], 4, s2)) return none();
    if (memcmp(kd.n, vd.n, sizeof kd.n) != 0 || memcmp(s1, s2, sizeof s1) != 0) return none();
    if (kd.n[0] != c.B || kd.n[1] != c.Hk || kd.n[2] < 1 || !fits(kd.n[2]) || kd.n[3] != c.d || s1[3] != 1)
      return none();
  }
  if (!ten(a[10], g_bf16, dev, 3, 1, &o) || memcmp(o.n, q.n, 3 * sizeof q.n[0]) != 0) return none();
  if (a[11] != Py_None &&
      (!ten(a[11], g_f32, dev, 2, 1, &lse) || lse.n[0] != c.B || lse.n[1] != q.n[1]))
    return none();
  if (!ten(a[12], g_f32, dev, 1, 1, &ws)) return none();
  const double scale = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) return none();
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_decode(q.p, &c, (const int*)lens.p, kd.p, vd.p, s1[0], s1[1], s1[2], (int)q.n[1], (int)kd.n[2],
                (float)scale, o.p, (float*)lse.p, (float*)ws.p, (size_t)ws.n[0] * 4, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

static PyObject* py_setup(PyObject* self, PyObject* args) {
  PyObject* o[7];
  Py_ssize_t append, gather, decode;
  if (!PyArg_ParseTuple(args, "OOOOOOOnnn", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6], &append,
                        &gather, &decode))
    return NULL;
  if (!PyType_Check(o[0])) {
    PyErr_SetString(PyExc_TypeError, "setup: the first argument is the tensor type");
    return NULL;
  }
  PyObject** to[7] = {&g_tensor, &g_bf16, &g_f32, &g_i32, &g_u8, &g_device, &g_stream};
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(o[i]);
    Py_XSETREF(*to[i], o[i]);
  }
  memcpy(&f_append, &append, sizeof append);
  memcpy(&f_gather, &gather, sizeof gather);
  memcpy(&f_decode, &decode, sizeof decode);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, NULL},
    {"append", (PyCFunction)(void (*)(void))py_append, METH_FASTCALL, NULL},
    {"gather", (PyCFunction)(void (*)(void))py_gather, METH_FASTCALL, NULL},
    {"decode", (PyCFunction)(void (*)(void))py_decode, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_py", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_paged_py(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  if (!s_dtype || !s_get_device || !s_is_contiguous || !s_data_ptr || !s_shape || !s_stride) return NULL;
  return PyModule_Create(&module);
}
