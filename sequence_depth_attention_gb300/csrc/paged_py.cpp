// The paged calls' arguments, marshalled by a Python extension: what binding.py
// does for tensors that are as the calls want them, without its time (an append
// of one token 3.7 us a call instead of 11.7, a decode of 701 rows 6.6 instead
// of 13.7). Anything else than that (a wrong type, a stream of its own) returns
// None, and binding.py goes through its own checks and says what is wrong.
//
//   setup(Tensor, device, stream, append, gather, decode, decode_workspace_bytes)
//       the tensor type, two callables (the current device, and the handle of
//       a device's current stream), and the addresses of the library's functions
//   more(prefill, prefill_workspace_bytes, means, select, selected)
//       the addresses of the functions that came later
//   append(...), gather(...), decode(...), prefill(...), means(...), select(...), selected(...)
//       the call's outputs, allocated where they are None; its status where
//       that is not 0; or None
#define PY_SSIZE_T_CLEAN
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>

#include "moda.h"

namespace {

PyObject *g_tensor, *g_device, *g_stream;
decltype(&moda_kv_append) f_append;
decltype(&moda_kv_gather) f_gather;
decltype(&moda_decode_paged) f_decode;
decltype(&moda_decode_paged_workspace_bytes) f_workspace;
decltype(&moda_prefill_paged) f_prefill;
decltype(&moda_prefill_paged_workspace_bytes) f_prefill_workspace;
decltype(&moda_page_means) f_means;
decltype(&moda_select_pages) f_select;
decltype(&moda_decode_selected) f_selected;

// A tensor argument: where its data is, its sizes and strides (the tensor's
// own, alive for the call).
struct Ten {
  void* p = nullptr;
  at::IntArrayRef n, s;
};

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt, kU8 = at::kByte;

// x: a tensor (not of a derived type) of this type and rank on device dev,
// contiguous if asked for.
bool ten(PyObject* x, at::ScalarType type, int64_t dev, size_t rank, bool contiguous, Ten* out) {
  if (reinterpret_cast<PyObject*>(Py_TYPE(x)) != g_tensor) return false;
  const at::Tensor& t = THPVariable_Unpack(x);
  if (t.scalar_type() != type || t.get_device() != dev || t.dim() != (int64_t)rank) return false;
  if (contiguous && !t.is_contiguous()) return false;
  out->n = t.sizes();
  out->s = t.strides();
  out->p = t.data_ptr();
  return true;
}

// An output: x where it is given and fits, else a new tensor in `made`, which
// must live as long as the call; device as of `like`.
bool output(PyObject* x, at::ScalarType type, at::IntArrayRef n, PyObject* like, int64_t dev, at::Tensor* made,
            Ten* out) {
  if (x != Py_None) return ten(x, type, dev, n.size(), true, out) && out->n == n;
  *made = at::empty(n, at::TensorOptions().dtype(type).device(THPVariable_Unpack(like).device()));
  out->n = made->sizes();
  out->p = made->data_ptr();
  return true;
}
// What the caller gets of an output: what it gave, the tensor made, or None.
PyObject* given(PyObject* x, const at::Tensor& made) {
  if (made.defined()) return THPVariable_Wrap(made);
  Py_INCREF(x);
  return x;
}
// The outputs, or the status of a call that failed; null where Python has none.
PyObject* result(moda_status st, PyObject* a, const at::Tensor& made_a, PyObject* b, const at::Tensor& made_b) {
  if (st != MODA_OK) return PyLong_FromLong(st);
  PyObject* x = given(a, made_a);
  PyObject* y = x ? given(b, made_b) : nullptr;
  PyObject* r = y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

bool fits(int64_t x) { return x <= INT32_MAX; }

bool current(int64_t* dev, moda_stream_t* stream) {
  PyObject* d = PyObject_CallNoArgs(g_device);
  if (!d) return false;
  *dev = PyLong_AsLongLong(d);
  PyObject* s = PyObject_CallOneArg(g_stream, d);
  Py_DECREF(d);
  if (!s) return false;
  *stream = (moda_stream_t)PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

// table: null where the call has none.
bool cache_of(PyObject* k, PyObject* v, PyObject* table, PyObject* ks, PyObject* vs, int64_t dev,
              moda_paged_kv* c) {
  const bool mx4 = ks != Py_None || vs != Py_None;
  const at::ScalarType type = mx4 ? kU8 : kBf16;
  Ten tk, tv, tt, a, b;
  if (!ten(k, type, dev, 4, true, &tk) || !ten(v, type, dev, 4, true, &tv)) return false;
  if (tk.n != tv.n || !fits(tk.n[0]) || !fits(tk.n[1]) || !fits(tk.n[2]) || !fits(2 * tk.n[3])) return false;
  c->B = 0;
  c->max_pages = 1;
  if (table) {
    if (!ten(table, kI32, dev, 2, true, &tt) || !fits(tt.n[0]) || !fits(tt.n[1])) return false;
    c->B = (int)tt.n[0];
    c->max_pages = (int)tt.n[1];
  }
  c->format = mx4 ? MODA_KV_MX4 : MODA_KV_BF16;
  c->num_pages = (int)tk.n[0];
  c->Hk = (int)tk.n[1];
  c->page_size = (int)tk.n[2];
  c->d = (int)tk.n[3] * (mx4 ? 2 : 1);
  c->k = tk.p;
  c->v = tv.p;
  c->block_table = (const int*)tt.p;
  if (mx4) {
    if (!ten(ks, kU8, dev, 4, true, &a) || !ten(vs, kU8, dev, 4, true, &b) || a.n != b.n) return false;
    if (a.n.slice(0, 3) != tk.n.slice(0, 3) || a.n[3] != c->d / 32) return false;
  }
  c->k_scale = a.p;
  c->v_scale = b.p;
  return true;
}

// Rows [N, H, d] with dense tokens (H < 0: any number); their distance.
bool rows(PyObject* x, int64_t dev, int64_t N, int64_t H, int64_t d, Ten* out, long long* stride) {
  if (!ten(x, kBf16, dev, 3, false, out) || out->n[0] != N || out->n[2] != d) return false;
  if ((H >= 0 && out->n[1] != H) || !fits(out->n[1])) return false;
  if (out->s[2] != 1 || (out->s[1] != d && out->n[1] > 1)) return false;
  *stride = N > 1 ? out->s[0] : out->n[1] * d;
  return true;
}

// seq and pos of at least one token.
bool tokens(PyObject* seq, PyObject* pos, int64_t dev, Ten* s, Ten* p) {
  return ten(seq, kI32, dev, 1, true, s) && ten(pos, kI32, dev, 1, true, p) && s->n == p->n && s->n[0] > 0 &&
         fits(s->n[0]);
}

// The calls: null where the arguments are not the plain case.
// (q, k, v, k_pages, v_pages, table, seq, pos, rope, interleaved, k_scales, v_scales, q_out, k_out, want_k_out)
PyObject* append(PyObject* const* a) {
  int64_t dev;
  long long qs = 0, ks, vs;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, k, v, seq, pos, rope, qo, ko;
  at::Tensor made_q, made_k;
  if (!current(&dev, &stream) || !cache_of(a[3], a[4], a[5], a[10], a[11], dev, &c)) return nullptr;
  if (!tokens(a[6], a[7], dev, &seq, &pos)) return nullptr;
  const int64_t N = seq.n[0];
  const bool queries = a[0] != Py_None, turn = a[8] != Py_None;
  if (queries ? !rows(a[0], dev, N, -1, c.d, &q, &qs) : a[12] != Py_None) return nullptr;
  if (!rows(a[1], dev, N, c.Hk, c.d, &k, &ks) || !rows(a[2], dev, N, c.Hk, c.d, &v, &vs)) return nullptr;
  if (turn && (!ten(a[8], kF32, dev, 2, true, &rope) || !fits(rope.n[0]) || !fits(rope.n[1]))) return nullptr;
  const int inter = PyObject_IsTrue(a[9]);
  if (inter < 0 || !PyBool_Check(a[14])) return nullptr;
  if (queries && !output(a[12], kBf16, q.n, a[0], dev, &made_q, &qo)) return nullptr;
  if ((a[13] != Py_None || a[14] == Py_True) && !output(a[13], kBf16, k.n, a[1], dev, &made_k, &ko))
    return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_append(q.p, k.p, v.p, qs, ks, vs, (const float*)rope.p, turn ? (int)rope.n[0] : 0,
                turn ? (int)rope.n[1] : 0, inter, (const int*)seq.p, (const int*)pos.p, (int)N,
                queries ? (int)q.n[1] : 0, &c, qo.p, ko.p, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[12], made_q, a[13], made_k);
}

// (k_pages, v_pages, table, seq, pos, k_scales, v_scales, k, v)
PyObject* gather(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten seq, pos, k, v;
  at::Tensor made_k, made_v;
  if (!current(&dev, &stream) || !cache_of(a[0], a[1], a[2], a[5], a[6], dev, &c)) return nullptr;
  if (!tokens(a[3], a[4], dev, &seq, &pos)) return nullptr;
  const int64_t n[3] = {seq.n[0], c.Hk, c.d};
  if (!output(a[7], kBf16, n, a[0], dev, &made_k, &k) || !output(a[8], kBf16, n, a[0], dev, &made_v, &v))
    return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_gather(&c, (const int*)seq.p, (const int*)pos.p, (int)seq.n[0], k.p, v.p, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[7], made_k, a[8], made_v);
}

// (q, k_pages, v_pages, table, seq_lens, scale, kd, vd, k_scales, v_scales, o, lse, workspace, want_lse)
PyObject* decode(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, lens, kd, vd, o, lse, ws;
  at::Tensor made_o, made_lse, made_ws;
  if (!current(&dev, &stream) || !cache_of(a[1], a[2], a[3], a[8], a[9], dev, &c)) return nullptr;
  if (!ten(a[0], kBf16, dev, 3, true, &q) || !ten(a[4], kI32, dev, 1, true, &lens)) return nullptr;
  if (c.B < 1 || q.n[0] != c.B || q.n[2] != c.d || !fits(q.n[1]) || lens.n[0] != c.B) return nullptr;
  long long s[3] = {0, 0, 0};
  int L = 0;
  if (a[6] != Py_None || a[7] != Py_None) {
    if (!ten(a[6], kBf16, dev, 4, false, &kd) || !ten(a[7], kBf16, dev, 4, false, &vd)) return nullptr;
    if (kd.n != vd.n || kd.s != vd.s || kd.n[0] != c.B || kd.n[1] != c.Hk || kd.n[3] != c.d) return nullptr;
    if (kd.s[3] != 1 || kd.n[2] < 1 || !fits(kd.n[2])) return nullptr;
    L = (int)kd.n[2];
    for (int i = 0; i < 3; ++i) s[i] = kd.s[i];
  }
  const double scale = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred() || !PyBool_Check(a[13])) return nullptr;
  const int Hq = (int)q.n[1];
  const int64_t heads[2] = {c.B, Hq};
  if (!output(a[10], kBf16, q.n, a[0], dev, &made_o, &o)) return nullptr;
  if ((a[11] != Py_None || a[13] == Py_True) && !output(a[11], kF32, heads, a[0], dev, &made_lse, &lse))
    return nullptr;
  if (a[12] != Py_None) {
    if (!ten(a[12], kF32, dev, 1, true, &ws)) return nullptr;
  } else {
    const int64_t need[1] = {std::max<int64_t>(4, (int64_t)(f_workspace(Hq, c.Hk, c.d) / 4))};
    if (!output(Py_None, kF32, need, a[0], dev, &made_ws, &ws)) return nullptr;
  }
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_decode(q.p, &c, (const int*)lens.p, kd.p, vd.p, s[0], s[1], s[2], Hq, L, (float)scale, o.p,
                (float*)lse.p, (float*)ws.p, (size_t)ws.n[0] * 4, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[10], made_o, a[11], made_lse);
}

// kd and vd of one shape, which is n with -1 where L stands, and strides: L and the first
// three strides; L = 0 where both are None.
bool depth(PyObject* k, PyObject* v, int64_t dev, const int64_t (&n)[4], Ten* kd, Ten* vd, int* L, long long (&s)[3]) {
  *L = 0;
  s[0] = s[1] = s[2] = 0;
  if (k == Py_None && v == Py_None) return true;
  if (!ten(k, kBf16, dev, 4, false, kd) || !ten(v, kBf16, dev, 4, false, vd)) return false;
  if (kd->n != vd->n || kd->s != vd->s || kd->s[3] != 1) return false;
  for (int i = 0; i < 4; ++i) {
    if (kd->n[i] < 1 || !fits(kd->n[i]) || (n[i] >= 0 && kd->n[i] != n[i])) return false;
    if (n[i] < 0) *L = (int)kd->n[i];
  }
  for (int i = 0; i < 3; ++i) s[i] = kd->s[i];
  return true;
}

// o [N, Hq, d], lse [N, Hq] and the workspace of an attention call.
bool attention_outputs(PyObject* o, PyObject* lse, PyObject* workspace, PyObject* want_lse, at::IntArrayRef q,
                       size_t workspace_bytes, PyObject* like, int64_t dev, at::Tensor (&made)[3], Ten (&out)[3]) {
  if (!PyBool_Check(want_lse) || !output(o, kBf16, q, like, dev, &made[0], &out[0])) return false;
  if ((lse != Py_None || want_lse == Py_True) && !output(lse, kF32, q.slice(0, 2), like, dev, &made[1], &out[1]))
    return false;
  if (workspace != Py_None) return ten(workspace, kF32, dev, 1, true, &out[2]);
  const int64_t need[1] = {std::max<int64_t>(4, (int64_t)(workspace_bytes / 4))};
  return output(Py_None, kF32, need, like, dev, &made[2], &out[2]);
}

// (q, k_pages, v_pages, table, q_starts, seq_lens, scale, kd, vd, k_scales, v_scales, o, lse, workspace, want_lse)
PyObject* prefill(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, starts, lens, kd, vd, out[3];
  at::Tensor made[3];
  long long qs, s[3];
  int L;
  if (!f_prefill || !current(&dev, &stream) || !cache_of(a[1], a[2], a[3], a[9], a[10], dev, &c)) return nullptr;
  if (!ten(a[4], kI32, dev, 1, true, &starts) || !ten(a[5], kI32, dev, 1, true, &lens)) return nullptr;
  if (c.B < 1 || lens.n[0] != c.B || starts.n[0] != (int64_t)c.B + 1) return nullptr;
  if (!ten(a[0], kBf16, dev, 3, false, &q) || q.n[0] < 1 || !fits(q.n[0])) return nullptr;
  if (!rows(a[0], dev, q.n[0], -1, c.d, &q, &qs)) return nullptr;
  const int64_t shape[4] = {-1, q.n[0], c.Hk, c.d};
  if (!depth(a[7], a[8], dev, shape, &kd, &vd, &L, s)) return nullptr;
  const double scale = PyFloat_AsDouble(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const int Hq = (int)q.n[1];
  if (!attention_outputs(a[11], a[12], a[13], a[14], q.n, f_prefill_workspace(Hq, c.Hk, c.d), a[0], dev, made, out))
    return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_prefill(q.p, qs, &c, (const int*)starts.p, (const int*)lens.p, kd.p, vd.p, s[0], s[1], s[2], (int)q.n[0], Hq,
                 L, (float)scale, out[0].p, (float*)out[1].p, (float*)out[2].p, (size_t)out[2].n[0] * 4, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[11], made[0], a[12], made[1]);
}

// (k_pages, v_pages, table, seq, pos, means, k_scales, v_scales)
PyObject* means(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten seq, pos, m;
  if (!f_means || !current(&dev, &stream) || !cache_of(a[0], a[1], a[2], a[6], a[7], dev, &c)) return nullptr;
  if (!tokens(a[3], a[4], dev, &seq, &pos) || !ten(a[5], kBf16, dev, 3, true, &m)) return nullptr;
  if (m.n[0] != c.num_pages || m.n[1] != c.Hk || m.n[2] != c.d) return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_means(&c, (const int*)seq.p, (const int*)pos.p, (int)seq.n[0], m.p, stream);
  Py_END_ALLOW_THREADS
  if (st != MODA_OK) return PyLong_FromLong(st);
  return PyTuple_Pack(1, a[5]);
}

// (q, means, k_pages, v_pages, table, seq, pos, S, sink, recent, k_scales, v_scales, pages, rows)
PyObject* select(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, m, seq, pos, pages, rows_;
  at::Tensor made_pages, made_rows;
  if (!f_select || !current(&dev, &stream) || !cache_of(a[2], a[3], a[4], a[10], a[11], dev, &c)) return nullptr;
  if (!tokens(a[5], a[6], dev, &seq, &pos) || !ten(a[0], kBf16, dev, 3, true, &q) ||
      !ten(a[1], kBf16, dev, 3, true, &m))
    return nullptr;
  if (q.n[0] != seq.n[0] || q.n[2] != c.d || !fits(q.n[1])) return nullptr;
  if (m.n[0] != c.num_pages || m.n[1] != c.Hk || m.n[2] != c.d) return nullptr;
  long n[3];
  for (int i = 0; i < 3; ++i) {
    if (!PyLong_CheckExact(a[7 + i])) return nullptr;
    n[i] = PyLong_AsLong(a[7 + i]);
    if (PyErr_Occurred() || n[i] < 0 || !fits(n[i])) return nullptr;
  }
  const int64_t shape[3] = {q.n[0], c.Hk, n[0]};
  if (!output(a[12], kI32, shape, a[0], dev, &made_pages, &pages) ||
      !output(a[13], kI32, at::IntArrayRef(shape, 2), a[0], dev, &made_rows, &rows_))
    return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_select(q.p, m.p, &c, (const int*)seq.p, (const int*)pos.p, (int)q.n[0], (int)q.n[1], (int)n[0], (int)n[1],
                (int)n[2], (int*)pages.p, (int*)rows_.p, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[12], made_pages, a[13], made_rows);
}

// (q, k_pages, v_pages, pages, rows, scale, kd, vd, k_scales, v_scales, o, lse, workspace, want_lse)
PyObject* selected(PyObject* const* a) {
  int64_t dev;
  moda_stream_t stream;
  moda_paged_kv c;
  Ten q, pages, rows_, kd, vd, out[3];
  at::Tensor made[3];
  long long s[3];
  int L;
  if (!f_selected || !current(&dev, &stream) || !cache_of(a[1], a[2], nullptr, a[8], a[9], dev, &c)) return nullptr;
  c.block_table = nullptr;
  if (!ten(a[0], kBf16, dev, 3, true, &q) || !ten(a[3], kI32, dev, 3, true, &pages) ||
      !ten(a[4], kI32, dev, 2, true, &rows_))
    return nullptr;
  if (q.n[0] < 1 || !fits(q.n[0]) || !fits(q.n[1]) || q.n[2] != c.d) return nullptr;
  if (pages.n[0] != q.n[0] || pages.n[1] != c.Hk || pages.n.slice(0, 2) != rows_.n || !fits(pages.n[2]))
    return nullptr;
  const int64_t shape[4] = {q.n[0], c.Hk, -1, c.d};
  if (!depth(a[6], a[7], dev, shape, &kd, &vd, &L, s)) return nullptr;
  const double scale = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const int Hq = (int)q.n[1];
  if (!attention_outputs(a[10], a[11], a[12], a[13], q.n, f_workspace(Hq, c.Hk, c.d), a[0], dev, made, out))
    return nullptr;
  moda_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f_selected(q.p, &c, (const int*)pages.p, (const int*)rows_.p, (int)q.n[0], (int)pages.n[2], kd.p, vd.p, s[0],
                  s[1], s[2], Hq, L, (float)scale, out[0].p, (float*)out[1].p, (float*)out[2].p,
                  (size_t)out[2].n[0] * 4, stream);
  Py_END_ALLOW_THREADS
  return result(st, a[10], made[0], a[11], made[1]);
}

template <PyObject* (*CALL)(PyObject* const*), int ARGS>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n == ARGS && g_tensor)
      if (PyObject* r = CALL(a)) return r;
  } catch (...) {  // a tensor without storage or no memory: binding.py meets it too
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

PyObject* setup(PyObject*, PyObject* args) {
  PyObject* o[3];
  Py_ssize_t append_at, gather_at, decode_at, workspace_at;
  if (!PyArg_ParseTuple(args, "OOOnnnn", &o[0], &o[1], &o[2], &append_at, &gather_at, &decode_at, &workspace_at))
    return nullptr;
  PyObject** to[3] = {&g_tensor, &g_device, &g_stream};
  for (int i = 0; i < 3; ++i) {
    Py_INCREF(o[i]);
    Py_XSETREF(*to[i], o[i]);
  }
  f_append = reinterpret_cast<decltype(f_append)>(append_at);
  f_gather = reinterpret_cast<decltype(f_gather)>(gather_at);
  f_decode = reinterpret_cast<decltype(f_decode)>(decode_at);
  f_workspace = reinterpret_cast<decltype(f_workspace)>(workspace_at);
  Py_RETURN_NONE;
}

PyObject* more(PyObject*, PyObject* args) {
  Py_ssize_t at[5];
  if (!PyArg_ParseTuple(args, "nnnnn", &at[0], &at[1], &at[2], &at[3], &at[4])) return nullptr;
  f_prefill = reinterpret_cast<decltype(f_prefill)>(at[0]);
  f_prefill_workspace = reinterpret_cast<decltype(f_prefill_workspace)>(at[1]);
  f_means = reinterpret_cast<decltype(f_means)>(at[2]);
  f_select = reinterpret_cast<decltype(f_select)>(at[3]);
  f_selected = reinterpret_cast<decltype(f_selected)>(at[4]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, nullptr},
                         {"more", more, METH_VARARGS, nullptr},
                         {"prefill", as_method(method<prefill, 15>), METH_FASTCALL, nullptr},
                         {"means", as_method(method<means, 8>), METH_FASTCALL, nullptr},
                         {"select", as_method(method<select, 14>), METH_FASTCALL, nullptr},
                         {"selected", as_method(method<selected, 14>), METH_FASTCALL, nullptr},
                         {"append", as_method(method<append, 15>), METH_FASTCALL, nullptr},
                         {"gather", as_method(method<gather, 9>), METH_FASTCALL, nullptr},
                         {"decode", as_method(method<decode, 14>), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_py", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_paged_py() { return PyModule_Create(&module); }
