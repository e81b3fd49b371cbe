/* pyargs.c -- CPython side of nk.py's calls that sit in a decode step: reads
 * the tensors' addresses, sizes and strides, checks them, and calls libnk.
 *
 * Written against the CPython C API alone (no torch headers): a tensor is any
 * object with torch's shape, dtype, stride(), get_device() and data_ptr().
 * Reading one costs about 0.3 us here against 0.9 us in Python, and a call
 * takes two to nine of them.  A refused argument raises ValueError; otherwise
 * the libnk status is returned for nk.py to raise. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "nk.h"

static struct {
  int (*norm_rope)(const nk_rope*, int32_t, const nk_rows*, int32_t, const nk_rows*, int32_t, const int32_t*, int32_t,
                   const nk_rows*, const nk_rows*, void*);
  int (*append_rope)(nk_pool*, int32_t, const int32_t*, const int32_t*, const int32_t*, const int32_t*, const nk_rope*,
                     const nk_rows*, const nk_rows*, const nk_rows*, int32_t, void*, int32_t, int32_t, void*);
  int (*shared)(const void*, int32_t, const nk_pool*, int32_t, const int32_t*, const int32_t*, const int32_t*,
                const int32_t*, int32_t, int32_t, float, void*, float*, int64_t, void*, size_t, void*);
  int (*verify)(const float*, int64_t, const float*, int64_t, const int32_t*, const int32_t*, const float*,
                const int32_t*, int32_t, int32_t, int32_t, int32_t*, int32_t*, int32_t*, void*);
  int (*diff_decode)(const void*, int32_t, const nk_pool*, int32_t, const int32_t*, const int32_t*, const int32_t*,
                     int32_t, int32_t, float, const nk_diff*, void*, float*, void*, size_t, void*);
  int (*diff_prefill)(const void*, int32_t, const nk_pool*, int32_t, const int32_t*, const int32_t*, const int32_t*,
                      const int32_t*, int32_t, int32_t, float, const nk_diff*, void*, float*, void*, size_t, void*);
  int (*residual_norm)(const nk_block_norm*, int32_t, int32_t, const void*, int64_t, const void*, int64_t, const void*,
                       int64_t, void*, int64_t, void*, int64_t, void*);
  int (*grow)(const nk_pool*, int32_t*, const int32_t*, const int32_t*, const int32_t*, const int32_t*, const int32_t*,
              int32_t*, int32_t*, const int32_t*, int32_t*, int32_t, int32_t, int32_t*, int32_t*, int64_t*, void*);
} lib;

static PyObject *n_shape, *n_dtype, *n_stride, *n_get_device, *n_data_ptr, *n_element_size;
static PyObject *t_bf16, *t_f32, *t_i32, *t_i64;

typedef struct {
  int nd;
  int64_t size[4], stride[4];
  void* ptr;
} Tensor;

static int ints(PyObject* tuple, int64_t* out, int* n) {
  if (!tuple) return 0;
  int ok = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) <= 4;
  *n = ok ? (int)PyTuple_GET_SIZE(tuple) : -1;
  for (int i = 0; ok && i < *n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
    if (out[i] == -1 && PyErr_Occurred()) ok = 0;
  }
  Py_DECREF(tuple);
  if (!ok && !PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "expected a tensor of at most four dimensions");
  return ok;
}

static int long_of(PyObject* v, long long* out) {
  if (!v) return 0;
  *out = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return !(*out == -1 && PyErr_Occurred());
}

static int refuse(const char* name, const char* what, PyObject* x) {
  PyObject *shape = PyObject_GetAttr(x, n_shape), *dtype = PyObject_GetAttr(x, n_dtype);
  PyErr_Clear();
  PyErr_Format(PyExc_ValueError, "%s: %s, got %S %S", name, what, dtype ? dtype : Py_None, shape ? shape : Py_None);
  Py_XDECREF(shape);
  Py_XDECREF(dtype);
  return 0;
}

/* Reads a tensor that has to be of `type` (NULL: any) on CUDA device `dev`. */
static int look(PyObject* x, const char* name, PyObject* type, long dev, Tensor* t) {
  PyObject* dtype = PyObject_GetAttr(x, n_dtype);
  if (!dtype) return 0;
  Py_DECREF(dtype); /* dtypes are objects for the life of the process */
  if (type && dtype != type) return refuse(name, type == t_bf16  ? "expected a bf16 tensor"
                                         : type == t_f32 ? "expected a float32 tensor"
                                         : type == t_i64 ? "expected an int64 tensor"
                                                         : "expected an int32 tensor", x);
  long long on, ptr;
  if (!long_of(PyObject_CallMethodNoArgs(x, n_get_device), &on)) return 0;
  if (on != dev) return refuse(name, on < 0 ? "expected a CUDA tensor" : "expected a tensor on the call's device", x);
  int nd;
  if (!ints(PyObject_GetAttr(x, n_shape), t->size, &t->nd) ||
      !ints(PyObject_CallMethodNoArgs(x, n_stride), t->stride, &nd) ||
      !long_of(PyObject_CallMethodNoArgs(x, n_data_ptr), &ptr))
    return 0;
  t->ptr = (void*)(intptr_t)ptr;
  return 1;
}

/* The same, contiguous (the stride of a dimension of size 1 says nothing) and
 * of the given sizes. */
static int plain(PyObject* x, const char* name, PyObject* type, long dev, int nd, const int64_t* size, Tensor* t) {
  if (!look(x, name, type, dev, t)) return 0;
  int ok = t->nd == nd;
  for (int i = 0; ok && i < nd; ++i) ok = t->size[i] == size[i];
  int64_t step = 1;
  for (int i = nd - 1; ok && i >= 0; --i) {
    ok = t->size[i] <= 1 || t->stride[i] == step;
    step *= t->size[i];
  }
  for (int i = 0; !ok && t->nd == nd && i < nd; ++i)
    if (size[i] == 0 && t->size[i] == 0) ok = 1; /* nothing in it */
  return ok ? 1 : refuse(name, "expected a contiguous tensor of the call's sizes", x);
}

/* Head rows: [N, heads, D] or [B, T, heads, D] with a unit last stride and
 * tokens one stride apart. */
static int rows_of(PyObject* x, const char* name, long dev, Tensor* t, nk_rows* r) {
  if (!look(x, name, t_bf16, dev, t)) return 0;
  const int n = t->nd;
  if (n < 3 || n > 4 || (t->stride[n - 1] != 1 && t->size[n - 1] > 1))
    return refuse(name, "expected [..., heads, head_dim] with a unit last stride", x);
  int64_t token = t->stride[n - 3];
  if (n == 4 && t->size[0] > 1) {
    if (t->size[1] == 1) token = t->stride[0];
    else if (t->stride[0] != t->size[1] * token) return refuse(name, "expected tokens one stride apart", x);
  }
  /* the stride of a dimension of size 1 says nothing */
  const int one = t->size[0] == 1 && (n == 3 || t->size[1] == 1);
  r->ptr = t->ptr;
  r->token_stride = one ? 0 : token;
  r->head_stride = t->size[n - 2] > 1 ? t->stride[n - 2] : 0;
  return 1;
}

/* Scratch memory: a contiguous tensor of any type, or its address with *bytes
 * given. */
static int scratch(PyObject* x, long dev, void** ptr, size_t* bytes) {
  if (PyLong_Check(x)) {
    *ptr = PyLong_AsVoidPtr(x);
    return !(!*ptr && PyErr_Occurred());
  }
  Tensor t;
  long long each;
  if (!look(x, "workspace", NULL, dev, &t) || !plain(x, "workspace", NULL, dev, t.nd, t.size, &t) ||
      !long_of(PyObject_CallMethodNoArgs(x, n_element_size), &each))
    return 0;
  *ptr = t.ptr;
  *bytes = (size_t)each;
  for (int i = 0; i < t.nd; ++i) *bytes *= (size_t)t.size[i];
  return 1;
}

static int same_size(const Tensor* a, const Tensor* b, int upto) {
  if (a->nd != b->nd) return 0;
  for (int i = 0; i < upto; ++i)
    if (a->size[i] != b->size[i]) return 0;
  return 1;
}

static int want(Py_ssize_t got, Py_ssize_t n) {
  if (got == n) return 1;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, got);
  return 0;
}

/* A layer number that no pool has, for one that does not fit. */
static int32_t layer32(long layer) { return layer < 0 || layer > INT32_MAX ? -1 : (int32_t)layer; }

#define ADDRESS(o) PyLong_AsVoidPtr(o)
#define NONE(o) ((o) == Py_None)
#define CALL(rc, call)       \
  Py_BEGIN_ALLOW_THREADS     \
  rc = call;                 \
  Py_END_ALLOW_THREADS

/* (q, k, positions, q_out, k_out, rope address, weights' head_dim or 0, device, stream) */
static PyObject* norm_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, p, qo, ko;
  nk_rows rq, rk, oq, ok;
  if (!want(n, 9)) return NULL;
  const long hd = PyLong_AsLong(a[6]), dev = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return NULL; /* no call to Python with an error set */
  if (!rows_of(a[0], "q", dev, &q, &rq) || !rows_of(a[1], "k", dev, &k, &rk)) return NULL;
  const int D = q.nd - 1, lead = q.nd - 2;
  if (!same_size(&q, &k, lead) || k.size[D] != q.size[D] || (hd && hd != q.size[D]))
    return refuse("k", "expected the tokens and the head_dim of q and of the norm weights", a[1]), NULL;
  if (a[3] == a[0]) oq = rq;
  else if (!rows_of(a[3], "q_out", dev, &qo, &oq)) return NULL;
  else if (!same_size(&q, &qo, q.nd)) return refuse("q_out", "expected the sizes of q", a[3]), NULL;
  if (a[4] == a[1]) ok = rk;
  else if (!rows_of(a[4], "k_out", dev, &ko, &ok)) return NULL;
  else if (!same_size(&k, &ko, k.nd)) return refuse("k_out", "expected the sizes of k", a[4]), NULL;
  if (!plain(a[2], "positions", t_i32, dev, lead, q.size, &p)) return NULL;
  const int64_t N = lead == 1 ? q.size[0] : q.size[0] * q.size[1];
  const nk_rope* rope = ADDRESS(a[5]);
  void* stream = ADDRESS(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (N > INT32_MAX) return refuse("q", "expected fewer tokens", a[0]), NULL;
  int rc;
  CALL(rc, lib.norm_rope(rope, (int32_t)q.size[D], &rq, (int32_t)q.size[D - 1], &rk, (int32_t)k.size[D - 1], p.ptr,
                         (int32_t)N, &oq, &ok, stream))
  return PyLong_FromLong(rc);
}

/* (pool address, H, D, C, L, layer, tables, table_rows, write_pos, k, v, q or None, q_out or None, counts or None,
 *  rope address, weights' head_dim or 0, device, stream) */
static PyObject* append_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, k, v, qo, t, r, w, c;
  nk_rows rq, rk, rv;
  if (!want(n, 18)) return NULL;
  const int64_t H = PyLong_AsLong(a[1]), D = PyLong_AsLong(a[2]);
  const int64_t table[2] = {PyLong_AsLong(a[3]), PyLong_AsLong(a[4])};
  const long layer = PyLong_AsLong(a[5]), hd = PyLong_AsLong(a[15]), dev = PyLong_AsLong(a[16]);
  if (PyErr_Occurred()) return NULL;
  const int has_q = !NONE(a[11]);
  if (!rows_of(a[9], "k", dev, &k, &rk) || !rows_of(a[10], "v", dev, &v, &rv)) return NULL;
  if (k.nd != 4 || k.size[2] != H || k.size[3] != D || (hd && hd != D))
    return refuse("k", "expected [B, T, KV heads, head_dim] of the pool and the norm weights", a[9]), NULL;
  if (!same_size(&k, &v, 4)) return refuse("v", "expected the sizes of k", a[10]), NULL;
  if (has_q) {
    if (!rows_of(a[11], "q", dev, &q, &rq)) return NULL;
    if (!same_size(&q, &k, 2) || q.size[3] != D)
      return refuse("q", "expected the tokens and the head_dim of k", a[11]), NULL;
    if (!plain(a[12], "q_out", t_bf16, dev, 4, q.size, &qo)) return NULL;
  } else if (!NONE(a[12])) {
    PyErr_SetString(PyExc_ValueError, "q_out without q");
    return NULL;
  }
  if (!plain(a[6], "tables", t_i32, dev, 2, table, &t) || !plain(a[7], "table_rows", t_i32, dev, 1, k.size, &r) ||
      !plain(a[8], "write_pos", t_i32, dev, 1, k.size, &w))
    return NULL;
  c.ptr = NULL;
  if (!NONE(a[13]) && !plain(a[13], "counts", t_i32, dev, 1, k.size, &c)) return NULL;
  nk_pool* pool = ADDRESS(a[0]);
  const nk_rope* rope = ADDRESS(a[14]);
  void* stream = ADDRESS(a[17]);
  if (PyErr_Occurred()) return NULL;
  if (k.size[1] > INT32_MAX || k.size[0] > INT32_MAX) return refuse("k", "expected fewer tokens", a[9]), NULL;
  int rc;
  CALL(rc, lib.append_rope(pool, layer32(layer), t.ptr, r.ptr, w.ptr, c.ptr, rope, &rk, &rv, has_q ? &rq : NULL,
                           has_q ? (int32_t)q.size[2] : 0, has_q ? qo.ptr : NULL, (int32_t)k.size[0],
                           (int32_t)k.size[1], stream))
  return PyLong_FromLong(rc);
}

/* (pool address, D, C, L, layer, q, tables, table_rows, frontiers, shared_pages, scale, out, lse, share_from,
 *  workspace, device, stream), or the workspace's address and bytes for it */
static PyObject* shared_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, t, r, f, s, o, l;
  void* ws;
  size_t bytes = 0;
  const int given = n == 18; /* bytes of the workspace */
  if (!given && !want(n, 17)) return NULL;
  const Py_ssize_t at = 15 + given;
  const int64_t D = PyLong_AsLong(a[1]);
  const int64_t table[2] = {PyLong_AsLong(a[2]), PyLong_AsLong(a[3])};
  const long layer = PyLong_AsLong(a[4]), dev = PyLong_AsLong(a[at]);
  if (PyErr_Occurred()) return NULL;
  if (!look(a[5], "q", t_bf16, dev, &q)) return NULL;
  if (q.nd != 4 || q.size[3] != D) return refuse("q", "expected [B, T, query heads, head_dim] of the pool", a[5]), NULL;
  if (!plain(a[5], "q", t_bf16, dev, 4, q.size, &q) || !plain(a[6], "tables", t_i32, dev, 2, table, &t) ||
      !plain(a[7], "table_rows", t_i32, dev, 1, q.size, &r) || !plain(a[8], "frontiers", t_i32, dev, 1, q.size, &f) ||
      !plain(a[11], "out", t_bf16, dev, 4, q.size, &o) || !plain(a[12], "lse", t_f32, dev, 3, q.size, &l) ||
      !look(a[9], "shared_pages", t_i32, dev, &s))
    return NULL;
  for (int i = 0; i < s.nd; ++i)
    if (s.size[i] != 1) return refuse("shared_pages", "expected one value", a[9]), NULL;
  const double scale = PyFloat_AsDouble(a[10]);
  const long long from = PyLong_AsLongLong(a[13]);
  nk_pool* pool = ADDRESS(a[0]);
  void* stream = ADDRESS(a[at + 1]);
  if (given) bytes = PyLong_AsSize_t(a[15]);
  if (PyErr_Occurred() || !scratch(a[14], dev, &ws, &bytes)) return NULL;
  for (int i = 0; i < 3; ++i)
    if (q.size[i] > INT32_MAX) return refuse("q", "expected smaller sizes", a[5]), NULL;
  int rc;
  CALL(rc, lib.shared(q.ptr, (int32_t)q.size[2], pool, layer32(layer), t.ptr, r.ptr, f.ptr, s.ptr, (int32_t)q.size[0],
                      (int32_t)q.size[1], (float)scale, o.ptr, l.ptr, from, ws, bytes, stream))
  return PyLong_FromLong(rc);
}

/* Probability rows [B, n, V]: a row stride of at least V. */
static int prob_rows(PyObject* x, const char* name, long dev, const int64_t* size, Tensor* t, int64_t* stride) {
  if (!look(x, name, t_f32, dev, t)) return 0;
  const int64_t B = size[0], n = size[1], V = size[2];
  if (t->nd != 3 || t->size[0] != B || t->size[1] != n || t->size[2] != V)
    return refuse(name, "expected [B, K + 1, V] target and [B, K, V] draft probabilities", x);
  *stride = V;
  if (B * n > 1) *stride = n > 1 ? t->stride[1] : t->stride[0]; /* size 1 says nothing */
  if (n && ((V > 1 && t->stride[2] != 1) || *stride < V || (B > 1 && n > 1 && t->stride[0] != n * t->stride[1])))
    return refuse(name, "expected contiguous rows one stride apart", x);
  return 1;
}

/* (target, draft or None, tokens, draft_len or None, uniforms, frontiers or None, accepted, out, after or None,
 *  device, stream); the last three tensors are nk.py's own */
static PyObject* verify(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor p, q, x, dl, u, f;
  long long acc, out, after = 0;
  int64_t ps, qs = 0;
  if (!want(n, 11)) return NULL;
  const long dev = PyLong_AsLong(a[9]);
  if (PyErr_Occurred()) return NULL;
  if (!look(a[0], "target", t_f32, dev, &p)) return NULL;
  if (p.nd != 3 || p.size[1] < 1) return refuse("target", "expected [B, K + 1, V]", a[0]), NULL;
  const int64_t B = p.size[0], K = p.size[1] - 1, V = p.size[2];
  if (B > INT32_MAX || K > INT32_MAX || V > INT32_MAX) return refuse("target", "expected smaller sizes", a[0]), NULL;
  const int64_t size[3] = {B, K, V}, bk1[2] = {B, K + 1};
  if (!prob_rows(a[0], "target", dev, p.size, &p, &ps)) return NULL;
  q.ptr = dl.ptr = f.ptr = NULL;
  if (!NONE(a[1]) && !prob_rows(a[1], "draft", dev, size, &q, &qs)) return NULL;
  if (!plain(a[2], "tokens", t_i32, dev, 2, size, &x) || !plain(a[4], "uniforms", t_f32, dev, 2, bk1, &u)) return NULL;
  if (!NONE(a[3]) && !plain(a[3], "draft_len", t_i32, dev, 1, size, &dl)) return NULL;
  if (!NONE(a[5]) && (!plain(a[5], "frontiers", t_i32, dev, 1, size, &f) ||
                      !long_of(PyObject_CallMethodNoArgs(a[8], n_data_ptr), &after)))
    return NULL;
  if (!long_of(PyObject_CallMethodNoArgs(a[6], n_data_ptr), &acc) ||
      !long_of(PyObject_CallMethodNoArgs(a[7], n_data_ptr), &out))
    return NULL;
  void* stream = ADDRESS(a[10]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  CALL(rc, lib.verify(p.ptr, ps, K ? q.ptr : NULL, qs, K ? x.ptr : NULL, dl.ptr, u.ptr, f.ptr, (int32_t)B, (int32_t)K,
                      (int32_t)V, (int32_t*)acc, (int32_t*)out, (int32_t*)after, stream))
  return PyLong_FromLong(rc);
}

/* (prefill, pool address, D, C, L, layer, q, tables, table_rows, frontiers or prefix_len, None or chunk_len, scale,
 *  diff address, its heads, tokens (0: any) and norm size (0: any), out, lse, workspace, device, stream) */
static PyObject* diff(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor q, t, r, f, c, o, l;
  void* ws;
  size_t bytes = 0;
  if (!want(n, 21)) return NULL;
  const int prefill = PyObject_IsTrue(a[0]);
  if (prefill < 0) return NULL;
  const int64_t D = PyLong_AsLong(a[2]);
  const int64_t table[2] = {PyLong_AsLong(a[3]), PyLong_AsLong(a[4])};
  const long layer = PyLong_AsLong(a[5]), dev = PyLong_AsLong(a[19]);
  const int64_t heads = PyLong_AsLongLong(a[13]), tokens = PyLong_AsLongLong(a[14]), width = PyLong_AsLongLong(a[15]);
  if (PyErr_Occurred()) return NULL;
  if (!look(a[6], "q", t_bf16, dev, &q)) return NULL;
  if (q.nd != 4 || q.size[3] != D || q.size[2] % 2)
    return refuse("q", "expected [B, T, an even number of query heads, head_dim] of the pool", a[6]), NULL;
  for (int i = 0; i < 3; ++i)
    if (q.size[i] > INT32_MAX) return refuse("q", "expected smaller sizes", a[6]), NULL;
  if (heads != q.size[2] / 2 || (tokens && tokens != q.size[0] * q.size[1]) || (width && width != 2 * D))
    return refuse("q", "expected the heads, tokens and head_dim of lam and the norm weight", a[6]), NULL;
  const int64_t out[4] = {q.size[0], q.size[1], q.size[2] / 2, 2 * D};
  if (!plain(a[6], "q", t_bf16, dev, 4, q.size, &q) || !plain(a[7], "tables", t_i32, dev, 2, table, &t) ||
      !plain(a[8], "table_rows", t_i32, dev, 1, q.size, &r) ||
      !plain(a[9], prefill ? "prefix_len" : "frontiers", t_i32, dev, 1, q.size, &f) ||
      (prefill && !plain(a[10], "chunk_len", t_i32, dev, 1, q.size, &c)) ||
      !plain(a[16], "out", t_bf16, dev, 4, out, &o) || !plain(a[17], "lse", t_f32, dev, 3, q.size, &l))
    return NULL;
  const double scale = PyFloat_AsDouble(a[11]);
  nk_pool* pool = ADDRESS(a[1]);
  const nk_diff* d = ADDRESS(a[12]);
  void* stream = ADDRESS(a[20]);
  if (PyErr_Occurred() || !scratch(a[18], dev, &ws, &bytes)) return NULL;
  int rc;
  if (prefill) {
    CALL(rc, lib.diff_prefill(q.ptr, (int32_t)q.size[2], pool, layer32(layer), t.ptr, r.ptr, f.ptr, c.ptr,
                              (int32_t)q.size[0], (int32_t)q.size[1], (float)scale, d, o.ptr, l.ptr, ws, bytes, stream))
  } else {
    CALL(rc, lib.diff_decode(q.ptr, (int32_t)q.size[2], pool, layer32(layer), t.ptr, r.ptr, f.ptr, (int32_t)q.size[0],
                             (int32_t)q.size[1], (float)scale, d, o.ptr, l.ptr, ws, bytes, stream))
  }
  return PyLong_FromLong(rc);
}

/* Rows [N, dim] or [B, T, dim] with a unit last stride and tokens one stride
 * apart; *tokens and *stride are theirs. */
static int flat_rows(PyObject* x, const char* name, PyObject* type, long dev, Tensor* t, int64_t* tokens,
                     int64_t* stride) {
  if (!look(x, name, type, dev, t)) return 0;
  const int n = t->nd;
  if (n < 2 || n > 3 || (t->stride[n - 1] != 1 && t->size[n - 1] > 1))
    return refuse(name, "expected [..., dim] of two or three dimensions with a unit last stride", x);
  *tokens = n == 2 ? t->size[0] : t->size[0] * t->size[1];
  *stride = t->stride[n - 2];
  if (n == 3 && t->size[0] > 1) {
    if (t->size[1] == 1) *stride = t->stride[0];
    else if (t->stride[0] != t->size[1] * *stride) return refuse(name, "expected tokens one stride apart", x);
  }
  if (*tokens == 1) *stride = 0; /* the stride of a dimension of size 1 says nothing */
  return 1;
}

/* (norm address, weights' dim or 0, y or None, residual, gate or None, x_out or None, residual_out, fp32 residual,
 *  device, stream) */
static PyObject* residual_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor y, r, g, x, o;
  int64_t N, m, ys = 0, rs = 0, gs = 0, xs = 0, os = 0;
  if (!want(n, 10)) return NULL;
  const long dim = PyLong_AsLong(a[1]), dev = PyLong_AsLong(a[8]);
  const int wide = PyObject_IsTrue(a[7]);
  if (PyErr_Occurred()) return NULL;
  PyObject* type = wide ? t_f32 : t_bf16;
  if (!flat_rows(a[3], "residual", type, dev, &r, &N, &rs)) return NULL;
  const int D = r.nd - 1;
  if (dim && dim != r.size[D]) return refuse("residual", "expected the dim of the norm weights", a[3]), NULL;
  y.ptr = g.ptr = x.ptr = NULL;
  if (!NONE(a[2])) {
    if (!flat_rows(a[2], "y", t_bf16, dev, &y, &m, &ys)) return NULL;
    if (!same_size(&y, &r, r.nd)) return refuse("y", "expected the sizes of residual", a[2]), NULL;
  }
  if (!NONE(a[4])) {
    if (!look(a[4], "gate", t_bf16, dev, &g)) return NULL;
    if (g.nd == 1) {
      if (!plain(a[4], "gate", t_bf16, dev, 1, &r.size[D], &g)) return NULL;
    } else {
      if (!flat_rows(a[4], "gate", t_bf16, dev, &g, &m, &gs)) return NULL;
      if (!same_size(&g, &r, r.nd)) return refuse("gate", "expected the sizes of residual or [dim]", a[4]), NULL;
    }
  }
  if (!NONE(a[5])) {
    if (!flat_rows(a[5], "out", t_bf16, dev, &x, &m, &xs)) return NULL;
    if (!same_size(&x, &r, r.nd)) return refuse("out", "expected the sizes of residual", a[5]), NULL;
  }
  if (!flat_rows(a[6], "residual_out", type, dev, &o, &m, &os)) return NULL;
  if (!same_size(&o, &r, r.nd)) return refuse("residual_out", "expected the sizes of residual", a[6]), NULL;
  const nk_block_norm* norm = ADDRESS(a[0]);
  void* stream = ADDRESS(a[9]);
  if (PyErr_Occurred()) return NULL;
  if (N > INT32_MAX || r.size[D] > INT32_MAX) return refuse("residual", "expected smaller sizes", a[3]), NULL;
  int rc;
  CALL(rc, lib.residual_norm(norm, (int32_t)r.size[D], (int32_t)N, y.ptr, ys, g.ptr, gs, r.ptr, rs, o.ptr, os, x.ptr, xs,
                             stream))
  return PyLong_FromLong(rc);
}

/* (pool address, C, L, M, T, tables, table_rows, committed, counts or None, keep or None, mapped, mapped_out,
 *  free_pages, free_count, free_count_out, frontiers, positions or None, slots or None, device, stream) */
static PyObject* grow(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Tensor t, r, c, k, p, m, mo, fp, fc, fo, f, pos, slot;
  if (!want(n, 20)) return NULL;
  const int64_t C = PyLong_AsLong(a[1]), M = PyLong_AsLong(a[3]), T = PyLong_AsLong(a[4]), one = 1;
  const int64_t table[2] = {C, PyLong_AsLong(a[2])};
  const long dev = PyLong_AsLong(a[18]);
  if (PyErr_Occurred()) return NULL;
  if (!look(a[7], "committed", t_i32, dev, &c)) return NULL;
  if (c.nd != 1 || c.size[0] > INT32_MAX) return refuse("committed", "expected [B]", a[7]), NULL;
  const int64_t bt[2] = {c.size[0], T};
  k.ptr = p.ptr = pos.ptr = slot.ptr = NULL;
  if (!plain(a[7], "committed", t_i32, dev, 1, bt, &c) || !plain(a[5], "tables", t_i32, dev, 2, table, &t) ||
      !plain(a[6], "table_rows", t_i32, dev, 1, bt, &r) ||
      (!NONE(a[8]) && !plain(a[8], "counts", t_i32, dev, 1, bt, &k)) ||
      (!NONE(a[9]) && !plain(a[9], "keep", t_i32, dev, 1, table, &p)) ||
      !plain(a[10], "mapped", t_i32, dev, 1, table, &m) || !plain(a[11], "mapped_out", t_i32, dev, 1, table, &mo) ||
      !plain(a[12], "free_pages", t_i32, dev, 1, &M, &fp) || !plain(a[13], "free_count", t_i32, dev, 1, &one, &fc) ||
      !plain(a[14], "free_count_out", t_i32, dev, 1, &one, &fo) ||
      !plain(a[15], "frontiers", t_i32, dev, 1, bt, &f) ||
      (!NONE(a[16]) && !plain(a[16], "positions", t_i32, dev, 2, bt, &pos)) ||
      (!NONE(a[17]) && !plain(a[17], "slots", t_i64, dev, 2, bt, &slot)))
    return NULL;
  nk_pool* pool = ADDRESS(a[0]);
  void* stream = ADDRESS(a[19]);
  if (PyErr_Occurred()) return NULL;
  int rc;
  CALL(rc, lib.grow(pool, t.ptr, r.ptr, c.ptr, k.ptr, p.ptr, m.ptr, mo.ptr, fp.ptr, fc.ptr, fo.ptr, (int32_t)c.size[0],
                    T < 0 || T > INT32_MAX ? -1 : (int32_t)T, f.ptr, pos.ptr, slot.ptr, stream))
  return PyLong_FromLong(rc);
}

/* (the eight entry points' addresses, torch.bfloat16, torch.float32, torch.int32, torch.int64) */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!want(n, 12)) return NULL;
  void* f[8];
  for (int i = 0; i < 8; ++i) f[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return NULL;
  *(void**)&lib.norm_rope = f[0];
  *(void**)&lib.append_rope = f[1];
  *(void**)&lib.shared = f[2];
  *(void**)&lib.verify = f[3];
  *(void**)&lib.diff_decode = f[4];
  *(void**)&lib.diff_prefill = f[5];
  *(void**)&lib.residual_norm = f[6];
  *(void**)&lib.grow = f[7];
  t_bf16 = Py_NewRef(a[8]);
  t_f32 = Py_NewRef(a[9]);
  t_i32 = Py_NewRef(a[10]);
  t_i64 = Py_NewRef(a[11]);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, NULL},
    {"append_rope", (PyCFunction)(void (*)(void))append_rope, METH_FASTCALL, NULL},
    {"shared_decode", (PyCFunction)(void (*)(void))shared_decode, METH_FASTCALL, NULL},
    {"verify", (PyCFunction)(void (*)(void))verify, METH_FASTCALL, NULL},
    {"diff", (PyCFunction)(void (*)(void))diff, METH_FASTCALL, NULL},
    {"residual_norm", (PyCFunction)(void (*)(void))residual_norm, METH_FASTCALL, NULL},
    {"grow", (PyCFunction)(void (*)(void))grow, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pyargs", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pyargs(void) {
  n_shape = PyUnicode_InternFromString("shape");
  n_dtype = PyUnicode_InternFromString("dtype");
  n_stride = PyUnicode_InternFromString("stride");
  n_get_device = PyUnicode_InternFromString("get_device");
  n_data_ptr = PyUnicode_InternFromString("data_ptr");
  n_element_size = PyUnicode_InternFromString("element_size");
  if (!n_shape || !n_dtype || !n_stride || !n_get_device || !n_data_ptr || !n_element_size) return NULL;
  return PyModule_Create(&module);
}
