/* Marshalling of the mixer calls in C (CPython extension module _fast).
 *
 * A decode step's kernels run for 3 to 10 us; reading their dozen tensors'
 * sizes, strides and addresses from Python took 20 us a call, in C it takes 3
 * to 4. The functions here take the arguments of the functions of the same
 * name in ops.py, check that everything is as the plain case has it -- tensor
 * types, layouts, sizes, all on the current device -- and make the call of
 * libcconv.so on the current stream. They return its status, or None where
 * anything is not plain; ops.py then takes its own way, which either serves the
 * case or raises what is wrong with it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <dlfcn.h>

#include "cconv.h"

enum { F32 = 0, BF16 = 1, I32 = 2, U8 = 3, B8 = 4, F8 = 5, F8S = 6, MIN_DT = 5, NDT = 7 };
/* float32, bfloat16, int32, uint8, bool (flags may be either), and of a cache in 8 bits
 * float8_e4m3fn, float8_e8m0fnu (scales may be that or uint8) */
static PyObject* dtypes[NDT];
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
static PyObject* raw_stream; /* device index -> cudaStream_t as an int */
static PyObject* cur_device; /* () -> index of the current device */
static PyObject* new_bytes;  /* (tensor, n) -> n bytes beside it */

static int (*p_fwd)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*,
                    int64_t, const void*, int64_t, const float*, const float*, gdn_state_t,
                    const int32_t*, const int32_t*, const uint8_t*, int32_t, int32_t, int32_t,
                    int32_t, int32_t, int32_t, float, int32_t, int32_t, void*, int64_t, int32_t*,
                    cconv_stream_t);
static int (*p_upd)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*,
                    int64_t, const void*, int64_t, const float*, const float*, gdn_state_t,
                    const int32_t*, int32_t, int32_t, const int32_t*, const uint8_t*, int32_t,
                    int32_t, int32_t, int32_t, float, int32_t, int32_t, void*, int64_t, int32_t*,
                    cconv_stream_t);
static int (*p_norm)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*,
                     const void*, float, const float*, int32_t, int32_t, int32_t, const int32_t*,
                     kv_cache_t, const int32_t*, int32_t, int32_t, int32_t, void*, int64_t,
                     int32_t*, cconv_stream_t);
static int (*p_attn)(const void*, int64_t, kv_cache_t, const int32_t*, int64_t, int32_t,
                     const int32_t*, int32_t, int32_t, int32_t, float, int32_t, void*, int64_t,
                     float*, void*, int64_t, int32_t*, cconv_stream_t);

static int (*p_norm_q8)(const void*, int64_t, const void*, int64_t, const void*, int64_t,
                        const void*, const void*, float, const float*, int32_t, int32_t, int32_t,
                        const int32_t*, kv_cache_q8_t, const int32_t*, int32_t, int32_t, int32_t,
                        void*, int64_t, int32_t*, cconv_stream_t);
static int (*p_read_q8)(kv_cache_q8_t, const int32_t*, int32_t, int32_t, void*, int64_t, void*,
                        int64_t, int32_t*, cconv_stream_t);
static int (*p_attn_q8)(const void*, int64_t, kv_cache_q8_t, const int32_t*, int64_t, int32_t,
                        const int32_t*, int32_t, int32_t, int32_t, float, int32_t, void*, int64_t,
                        float*, void*, int64_t, int32_t*, cconv_stream_t);
static int (*p_shared)(const void*, int64_t, kv_cache_t, const int32_t*, int64_t, int32_t,
                       const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t, int32_t,
                       int32_t, float, int32_t, void*, int64_t, float*, void*, int64_t, int32_t*,
                       cconv_stream_t);
static int (*p_shared_q8)(const void*, int64_t, kv_cache_q8_t, const int32_t*, int64_t, int32_t,
                          const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t,
                          int32_t, int32_t, float, int32_t, void*, int64_t, float*, void*, int64_t,
                          int32_t*, cconv_stream_t);
static int64_t (*p_need)(int32_t, int32_t, int32_t, int32_t, int32_t);
static int64_t (*p_need_shared)(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t);

typedef struct {
  void* p;
  int nd, dt;             /* nd < 0: None */
  int64_t n[4], s[4];
} Ten;

/* 1: a CUDA tensor of at most 4 dimensions and a known type, or None; 0: not. *dev is the
 * device of the call's tensors, -1 before the first one: another device is not plain. */
static int get(PyObject* o, Ten* t, int* dev) {
  t->p = NULL;
  t->nd = -1;
  t->dt = -1;
  if (o == Py_None) return 1;
  PyObject* d = PyObject_GetAttr(o, s_dtype);
  if (!d) return 0;
  for (int i = 0; i < NDT; ++i)
    if (d == dtypes[i]) t->dt = i;
  Py_DECREF(d);
  if (t->dt < 0) return 0;
  PyObject* c = PyObject_CallMethodNoArgs(o, s_get_device);
  if (!c) return 0;
  const long on = PyLong_AsLong(c);
  Py_DECREF(c);
  if (on < 0 || (*dev >= 0 && on != *dev)) return 0; /* (a host tensor: -1) */
  *dev = (int)on;
  PyObject* sh = PyObject_GetAttr(o, s_shape);
  if (!sh) return 0;
  PyObject* st = PyObject_CallMethodNoArgs(o, s_stride);
  int ok = st && PyTuple_Check(sh) && PyTuple_Check(st) && PyTuple_GET_SIZE(sh) <= 4 &&
           PyTuple_GET_SIZE(sh) == PyTuple_GET_SIZE(st);
  if (ok) {
    t->nd = (int)PyTuple_GET_SIZE(sh);
    for (int i = 0; i < t->nd; ++i) {
      t->n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(sh, i));
      t->s[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    }
  }
  Py_DECREF(sh);
  Py_XDECREF(st);
  if (!ok || PyErr_Occurred()) return 0;
  PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!p) return 0;
  t->p = PyLong_AsVoidPtr(p);
  Py_DECREF(p);
  return !PyErr_Occurred();
}

/* A required tensor of this type. */
static int need(PyObject* o, Ten* t, int dt, int* dev) {
  return get(o, t, dev) && t->nd >= 0 && t->dt == dt;
}
/* An optional one. */
static int maybe(PyObject* o, Ten* t, int dt, int* dev) {
  return get(o, t, dev) && (t->nd < 0 || t->dt == dt);
}
/* Optional flags; required scales of a cache in 8 bits. */
static int flags(PyObject* o, Ten* t, int* dev) {
  return get(o, t, dev) && (t->nd < 0 || t->dt == U8 || t->dt == B8);
}
static int scales(PyObject* o, Ten* t, int* dev) {
  return get(o, t, dev) && t->nd >= 0 && (t->dt == U8 || t->dt == F8S);
}

/* [rows, heads, dim] with contiguous rows; *rs = row stride. */
static int heads(const Ten* t, int64_t rows, int64_t h, int64_t d, int64_t* rs) {
  if (t->nd != 3 || t->s[2] != 1 || (t->s[1] != t->n[2] && t->n[1] > 1) || t->n[0] < rows ||
      t->n[1] != h || t->n[2] != d)
    return 0;
  *rs = t->n[0] > 1 || t->s[0] > h * d ? t->s[0] : h * d;
  return 1;
}
static int gates(const Ten* t, int64_t rows, int64_t h, int64_t* rs) {
  if (t->nd != 2 || t->n[0] < rows || t->n[1] != h || (h > 1 && t->s[1] != 1)) return 0;
  *rs = t->n[0] > 1 || t->s[0] > h ? t->s[0] : h;
  return 1;
}
static int vec(const Ten* t, int64_t n) {
  return t->nd == 1 && t->n[0] == n && (n <= 1 || t->s[0] == 1);
}
static int flat(const Ten* t) { return t->nd == 1 && (t->n[0] <= 1 || t->s[0] == 1); }

/* The current stream of device `dev`, which has to be the current device. */
static int stream_of(int dev, cconv_stream_t* st) {
  PyObject* d = PyObject_CallNoArgs(cur_device);
  if (!d) return 0;
  const long cur = PyLong_AsLong(d);
  PyObject* r = cur == dev && !PyErr_Occurred() ? PyObject_CallOneArg(raw_stream, d) : NULL;
  Py_DECREF(d);
  if (!r) return 0;
  *st = (cconv_stream_t)PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  return !PyErr_Occurred();
}

static PyObject* not_plain(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

typedef struct {
  Ten q, k, v, a, b, A, dtb, st, out, err;
  int64_t qs, ks, vs, as, bs, os, hk, hv, dk, dv;
  int dev;
  gdn_state_t pool;
  cconv_stream_t stream;
} Gdn;

/* args: q k v a b A_log dt_bias states at 0..7; g->dev is set */
static int gdn(PyObject* const* x, PyObject* out, PyObject* err, int64_t rows, Gdn* g) {
  int* const dev = &g->dev;
  if (!get(x[1], &g->k, dev) || g->k.nd != 3 || (g->k.dt != F32 && g->k.dt != BF16)) return 0;
  const int dt = g->k.dt;
  if (!need(x[0], &g->q, dt, dev) || !need(x[2], &g->v, dt, dev) ||
      !need(x[3], &g->a, dt, dev) || !need(x[4], &g->b, dt, dev) ||
      !need(x[5], &g->A, F32, dev) || !need(x[6], &g->dtb, F32, dev) ||
      !get(x[7], &g->st, dev) || !need(out, &g->out, dt, dev) || !maybe(err, &g->err, I32, dev))
    return 0;
  if (g->v.nd != 3 || g->st.nd != 4 || (g->st.dt != F32 && g->st.dt != BF16)) return 0;
  g->hk = g->k.n[1], g->dk = g->k.n[2], g->hv = g->v.n[1], g->dv = g->v.n[2];
  const int64_t* n = g->st.n;
  const int64_t* s = g->st.s;
  if (!heads(&g->q, rows, g->hk, g->dk, &g->qs) || !heads(&g->k, rows, g->hk, g->dk, &g->ks) ||
      !heads(&g->v, rows, g->hv, g->dv, &g->vs) || !heads(&g->out, rows, g->hv, g->dv, &g->os) ||
      !gates(&g->a, rows, g->hv, &g->as) || !gates(&g->b, rows, g->hv, &g->bs) ||
      !vec(&g->A, g->hv) || !vec(&g->dtb, g->hv) || n[1] != g->hv || n[2] != g->dk ||
      n[3] != g->dv || s[3] != 1 || s[2] != g->dv)
    return 0;
  const int64_t one = g->dk * g->dv, all = g->hv * one;
  g->pool.p = g->st.p;
  g->pool.s_slot = n[0] > 1 || s[0] > all ? s[0] : all;
  g->pool.s_head = g->hv > 1 || s[1] > one ? s[1] : one;
  g->pool.num_slots = (int32_t)n[0];
  g->pool.dtype = g->st.dt;
  return stream_of(g->dev, &g->stream);
}

/* q k v a b A_log dt_bias states state_idx cu_seqlens has_init scale out l2norm dev_err rows */
static PyObject* f_fwd(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  Gdn g;
  g.dev = -1;
  Ten idx, cu, hi;
  if (n != 16) return not_plain();
  const double scale = PyFloat_AsDouble(x[11]);
  const long l2 = PyObject_IsTrue(x[13]);
  if (PyErr_Occurred() || !need(x[8], &idx, I32, &g.dev) || !need(x[9], &cu, I32, &g.dev) ||
      !flags(x[10], &hi, &g.dev) || !flat(&idx) || !flat(&cu) || cu.n[0] != idx.n[0] + 1 ||
      (hi.nd >= 0 && (!flat(&hi) || hi.n[0] < idx.n[0])))
    return not_plain();
  Ten q;
  int64_t rows;
  if (x[15] == Py_None) {
    if (!get(x[0], &q, &g.dev) || q.nd != 3) return not_plain();
    rows = q.n[0];
  } else {
    rows = PyLong_AsLongLong(x[15]);
    if (PyErr_Occurred()) return not_plain();
  }
  if (!gdn(x, x[12], x[14], rows, &g)) return not_plain();
  return PyLong_FromLong(p_fwd(
      g.q.p, g.qs, g.k.p, g.ks, g.v.p, g.vs, g.a.p, g.as, g.b.p, g.bs, g.A.p, g.dtb.p, g.pool,
      idx.p, cu.p, hi.p, (int32_t)idx.n[0], (int32_t)rows, (int32_t)g.hk, (int32_t)g.hv,
      (int32_t)g.dk, (int32_t)g.dv, (float)scale, (int32_t)l2, g.k.dt, g.out.p, g.os, g.err.p,
      g.stream));
}

/* q k v a b A_log dt_bias states state_idx n_spec num_accepted has_init scale out l2norm dev_err */
static PyObject* f_upd(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  Gdn g;
  g.dev = -1;
  Ten idx, acc, hi;
  if (n != 16) return not_plain();
  const long ns = PyLong_AsLong(x[9]);
  const double scale = PyFloat_AsDouble(x[12]);
  const long l2 = PyObject_IsTrue(x[14]);
  if (PyErr_Occurred() || !need(x[8], &idx, I32, &g.dev) || !maybe(x[10], &acc, I32, &g.dev) ||
      !flags(x[11], &hi, &g.dev) || idx.nd < 1 || idx.nd > 2 || ns < 0)
    return not_plain();
  const int64_t B = idx.n[0], w = idx.nd == 2 ? idx.n[1] : 1;
  if (w != 1 + ns || (idx.nd == 2 && w > 1 && idx.s[1] != 1) || (B > 1 && idx.s[0] != w) ||
      (acc.nd >= 0 && (!flat(&acc) || acc.n[0] < B)) ||
      (hi.nd >= 0 && (!flat(&hi) || hi.n[0] < B)) || !gdn(x, x[13], x[15], B * w, &g))
    return not_plain();
  return PyLong_FromLong(p_upd(
      g.q.p, g.qs, g.k.p, g.ks, g.v.p, g.vs, g.a.p, g.as, g.b.p, g.bs, g.A.p, g.dtb.p, g.pool,
      idx.p, (int32_t)B, (int32_t)ns, acc.p, hi.p, (int32_t)g.hk, (int32_t)g.hv, (int32_t)g.dk,
      (int32_t)g.dv, (float)scale, (int32_t)l2, g.k.dt, g.out.p, g.os, g.err.p, g.stream));
}

static int cache(PyObject* ko, PyObject* vo, int dt, kv_cache_t* c, int* dev) {
  Ten k, v;
  if (!need(ko, &k, dt, dev) || !need(vo, &v, dt, dev) || k.nd != 4 || v.nd != 4 || k.s[3] != 1)
    return 0;
  for (int i = 0; i < 4; ++i)
    if (k.n[i] != v.n[i] || k.s[i] != v.s[i]) return 0;
  int64_t s[3];
  for (int i = 0; i < 3; ++i) s[i] = k.n[i] > 1 || k.s[i] > k.n[3] ? k.s[i] : k.n[3];
  c->k = k.p, c->v = v.p;
  c->s_page = s[0], c->s_token = s[1], c->s_head = s[2];
  c->num_pages = (int32_t)k.n[0], c->page_size = (int32_t)k.n[1];
  c->num_kv_heads = (int32_t)k.n[2], c->head_dim = (int32_t)k.n[3];
  c->dtype = dt;
  return 1;
}

/* k_cache v_cache k_scale v_scale at x[0..3] */
static int cache_q8(PyObject* const* x, kv_cache_q8_t* c, int* dev) {
  kv_cache_t p;
  Ten k, v;
  if (!cache(x[0], x[1], F8, &p, dev) || !scales(x[2], &k, dev) || !scales(x[3], &v, dev) ||
      k.nd != 3 || v.nd != 3)
    return 0;
  const int64_t n[3] = {p.num_pages, p.page_size, p.num_kv_heads};
  int64_t s[3];
  for (int i = 0; i < 3; ++i) {
    if (k.n[i] != n[i] || v.n[i] != n[i] || k.s[i] != v.s[i]) return 0;
    s[i] = n[i] > 1 || k.s[i] > 1 ? k.s[i] : 1;
  }
  c->k = p.k, c->v = p.v;
  c->s_page = p.s_page, c->s_token = p.s_token, c->s_head = p.s_head;
  c->k_scale = k.p, c->v_scale = v.p;
  c->c_page = s[0], c->c_token = s[1], c->c_head = s[2];
  c->num_pages = p.num_pages, c->page_size = p.page_size;
  c->num_kv_heads = p.num_kv_heads, c->head_dim = p.head_dim;
  return 1;
}

/* q k v q_weight k_weight eps cos_sin positions interleaved k_cache v_cache [k_scale v_scale]
 * slots q_out dev_err */
static PyObject* norm(PyObject* const* x, Py_ssize_t n, int q8) {
  Ten q, k, v, qw, kw, cs, pos, sl, out, err;
  kv_cache_t c = {0};
  kv_cache_q8_t c8 = {0};
  int dev = -1;
  int64_t qs, ks, vs, os;
  cconv_stream_t st;
  if (n != (q8 ? 16 : 14) || !get(x[0], &q, &dev) || q.nd != 3 || (q.dt != F32 && q.dt != BF16))
    return not_plain();
  const int dt = q.dt;
  const int64_t T = q.n[0], hq = q.n[1], D = q.n[2];
  const double eps = PyFloat_AsDouble(x[5]);
  const long il = PyObject_IsTrue(x[8]);
  PyObject* const* y = x + (q8 ? 13 : 11); /* slots q_out dev_err */
  if (PyErr_Occurred() || !(q8 ? cache_q8(x + 9, &c8, &dev) : cache(x[9], x[10], dt, &c, &dev)))
    return not_plain();
  const int64_t hkv = q8 ? c8.num_kv_heads : c.num_kv_heads;
  if ((q8 ? c8.head_dim : c.head_dim) != D || !need(x[1], &k, dt, &dev) ||
      !need(x[2], &v, dt, &dev) || !maybe(x[3], &qw, dt, &dev) || !maybe(x[4], &kw, dt, &dev) ||
      !need(x[6], &cs, F32, &dev) || !need(x[7], &pos, I32, &dev) || !need(y[0], &sl, I32, &dev) ||
      !need(y[1], &out, dt, &dev) || !maybe(y[2], &err, I32, &dev))
    return not_plain();
  if (!heads(&q, T, hq, D, &qs) || !heads(&k, T, hkv, D, &ks) || !heads(&v, T, hkv, D, &vs) ||
      !heads(&out, T, hq, D, &os) || (qw.nd >= 0 && !vec(&qw, D)) || (kw.nd >= 0 && !vec(&kw, D)) ||
      !flat(&pos) || !flat(&sl) || pos.n[0] < T || sl.n[0] < T || cs.nd != 2 ||
      (cs.n[1] > 1 && cs.s[1] != 1) || (cs.n[0] > 1 && cs.s[0] != cs.n[1]) ||
      (err.nd >= 0 && (err.nd != 1 || err.n[0] < 1)) || !stream_of(dev, &st))
    return not_plain();
  return PyLong_FromLong(
      q8 ? p_norm_q8(q.p, qs, k.p, ks, v.p, vs, qw.p, kw.p, (float)eps, cs.p, (int32_t)cs.n[0],
                     (int32_t)cs.n[1], (int32_t)il, pos.p, c8, sl.p, (int32_t)T, (int32_t)hq, dt,
                     out.p, os, err.p, st)
         : p_norm(q.p, qs, k.p, ks, v.p, vs, qw.p, kw.p, (float)eps, cs.p, (int32_t)cs.n[0],
                  (int32_t)cs.n[1], (int32_t)il, pos.p, c, sl.p, (int32_t)T, (int32_t)hq, dt,
                  out.p, os, err.p, st));
}
static PyObject* f_norm(PyObject* self, PyObject* const* x, Py_ssize_t n) { return norm(x, n, 0); }
static PyObject* f_norm_q8(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  return norm(x, n, 1);
}

/* k_cache v_cache k_scale v_scale slots k_out v_out dev_err */
static PyObject* f_read_q8(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  Ten sl, ko, vo, err;
  kv_cache_q8_t c;
  int dev = -1;
  int64_t ks, vs;
  cconv_stream_t st;
  if (n != 8 || !cache_q8(x, &c, &dev) || !need(x[4], &sl, I32, &dev) || !flat(&sl) ||
      !get(x[5], &ko, &dev) || ko.nd != 3 || (ko.dt != F32 && ko.dt != BF16) ||
      !need(x[6], &vo, ko.dt, &dev) || !maybe(x[7], &err, I32, &dev))
    return not_plain();
  const int64_t T = sl.n[0];
  if (!heads(&ko, T, c.num_kv_heads, c.head_dim, &ks) ||
      !heads(&vo, T, c.num_kv_heads, c.head_dim, &vs) ||
      (err.nd >= 0 && (err.nd != 1 || err.n[0] < 1)) || !stream_of(dev, &st))
    return not_plain();
  return PyLong_FromLong(p_read_q8(c, sl.p, (int32_t)T, ko.dt, ko.p, ks, vo.p, vs, err.p, st));
}

/* q k_cache v_cache [k_scale v_scale] block_table seq_lens [cu_groups prefix_lens] n_spec scale
 * out lse workspace dev_err */
static PyObject* attn(PyObject* const* x, Py_ssize_t n, int q8, int shared) {
  Ten q, tab, len, cu, pre, out, lse, ws, err;
  kv_cache_t c = {0};
  kv_cache_q8_t c8 = {0};
  int dev = -1;
  int64_t qs, os, G = 0;
  cconv_stream_t st;
  if (n != 11 + 2 * q8 + 2 * shared || !get(x[0], &q, &dev) || q.nd != 3 ||
      (q.dt != F32 && q.dt != BF16))
    return not_plain();
  PyObject* const* t = x + 3 + 2 * q8;  /* block_table seq_lens [cu_groups prefix_lens] */
  PyObject* const* y = t + 2 + 2 * shared; /* n_spec .. */
  const long ns = PyLong_AsLong(y[0]);
  const double scale = PyFloat_AsDouble(y[1]);
  if (PyErr_Occurred() || ns < 0 ||
      !(q8 ? cache_q8(x + 1, &c8, &dev) : cache(x[1], x[2], q.dt, &c, &dev)) ||
      !need(t[0], &tab, I32, &dev) || !need(t[1], &len, I32, &dev) ||
      !need(y[2], &out, q.dt, &dev) || !maybe(y[3], &lse, F32, &dev) ||
      !maybe(y[4], &ws, U8, &dev) || !maybe(y[5], &err, I32, &dev) || !flat(&len) ||
      (ws.nd >= 0 && !flat(&ws)) || (err.nd >= 0 && (err.nd != 1 || err.n[0] < 1)))
    return not_plain();
  if (shared) {
    if (!need(t[2], &cu, I32, &dev) || !need(t[3], &pre, I32, &dev) || !flat(&cu) || !flat(&pre) ||
        cu.n[0] != pre.n[0] + 1)
      return not_plain();
    G = pre.n[0];
  }
  const int64_t B = len.n[0], rows = B * (1 + ns);
  const int32_t hkv = q8 ? c8.num_kv_heads : c.num_kv_heads, D = q8 ? c8.head_dim : c.head_dim;
  const int32_t hq = (int32_t)q.n[1];
  if (q.n[2] != D || !heads(&q, rows, hq, D, &qs) || !heads(&out, rows, hq, D, &os) ||
      tab.nd != 2 || tab.n[0] < B || (tab.n[1] > 1 && tab.s[1] != 1) ||
      (lse.nd >= 0 && (lse.nd != 2 || lse.n[0] < rows || lse.n[1] != q.n[1] ||
                       (lse.n[1] > 1 && lse.s[1] != 1) || (lse.n[0] > 1 && lse.s[0] != q.n[1]))) ||
      !stream_of(dev, &st))
    return not_plain();
  const int64_t ts = tab.n[0] > 1 || tab.s[0] > tab.n[1] ? tab.s[0] : tab.n[1];
  const int32_t tw = (int32_t)tab.n[1], b = (int32_t)B, s = (int32_t)ns, g = (int32_t)G;
  PyObject* own = NULL; /* the call's workspace, if it brought none */
  if (ws.nd < 0) {
    const int64_t need = shared ? p_need_shared(b, g, s, hq, hkv, D) : p_need(b, s, hq, hkv, D);
    if (need < 0) return not_plain();
    own = PyObject_CallFunction(new_bytes, "OL", x[0], (long long)(need > 16 ? need : 16));
    if (!own) return NULL;
    if (!get(own, &ws, &dev) || ws.nd != 1) {
      Py_DECREF(own);
      return not_plain();
    }
  }
  int rc;
  if (!shared)
    rc = q8 ? p_attn_q8(q.p, qs, c8, tab.p, ts, tw, len.p, b, s, hq, (float)scale, q.dt, out.p, os,
                        lse.p, ws.p, ws.n[0], err.p, st)
            : p_attn(q.p, qs, c, tab.p, ts, tw, len.p, b, s, hq, (float)scale, q.dt, out.p, os,
                     lse.p, ws.p, ws.n[0], err.p, st);
  else
    rc = q8 ? p_shared_q8(q.p, qs, c8, tab.p, ts, tw, len.p, b, cu.p, pre.p, g, s, hq,
                          (float)scale, q.dt, out.p, os, lse.p, ws.p, ws.n[0], err.p, st)
            : p_shared(q.p, qs, c, tab.p, ts, tw, len.p, b, cu.p, pre.p, g, s, hq, (float)scale,
                       q.dt, out.p, os, lse.p, ws.p, ws.n[0], err.p, st);
  Py_XDECREF(own);
  return PyLong_FromLong(rc);
}
#define ATTN(name, q8, shared)                                                      \
  static PyObject* name(PyObject* self, PyObject* const* x, Py_ssize_t n) {         \
    return attn(x, n, q8, shared);                                                  \
  }
ATTN(f_attn, 0, 0)
ATTN(f_attn_q8, 1, 0)
ATTN(f_shared, 0, 1)
ATTN(f_shared_q8, 1, 1)

/* init(handle of libcconv.so, (float32, bfloat16, int32, uint8, bool[, float8_e4m3fn,
 *      float8_e8m0fnu: without them 8-bit caches are left to Python]), raw stream function,
 *      function (tensor, n) -> n bytes on its device and the current stream, current device
 *      function) */
static PyObject* f_init(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  if (n != 5 || !PyTuple_Check(x[1]) ||
      (PyTuple_GET_SIZE(x[1]) != MIN_DT && PyTuple_GET_SIZE(x[1]) != NDT)) {
    PyErr_SetString(PyExc_TypeError, "init(handle, dtypes, raw_stream, new_bytes, cur_device)");
    return NULL;
  }
  void* h = PyLong_AsVoidPtr(x[0]);
  if (PyErr_Occurred()) return NULL;
  *(void**)&p_fwd = dlsym(h, "gdn_fwd_varlen");
  *(void**)&p_upd = dlsym(h, "gdn_update");
  *(void**)&p_norm = dlsym(h, "attn_norm_rope_cache");
  *(void**)&p_attn = dlsym(h, "attn_decode");
  *(void**)&p_need = dlsym(h, "attn_decode_workspace_bytes");
  *(void**)&p_norm_q8 = dlsym(h, "attn_norm_rope_cache_q8");
  *(void**)&p_read_q8 = dlsym(h, "kv_cache_read_q8");
  *(void**)&p_attn_q8 = dlsym(h, "attn_decode_q8");
  *(void**)&p_shared = dlsym(h, "attn_decode_shared");
  *(void**)&p_shared_q8 = dlsym(h, "attn_decode_shared_q8");
  *(void**)&p_need_shared = dlsym(h, "attn_decode_shared_workspace_bytes");
  if (!p_fwd || !p_upd || !p_norm || !p_attn || !p_need || !p_norm_q8 || !p_read_q8 ||
      !p_attn_q8 || !p_shared || !p_shared_q8 || !p_need_shared) {
    PyErr_SetString(PyExc_RuntimeError, "libcconv.so lacks an entry point");
    return NULL;
  }
  for (int i = 0; i < NDT; ++i)
    Py_XSETREF(dtypes[i], i < PyTuple_GET_SIZE(x[1]) ? Py_NewRef(PyTuple_GET_ITEM(x[1], i)) : NULL);
  Py_XSETREF(raw_stream, Py_NewRef(x[2]));
  Py_XSETREF(new_bytes, Py_NewRef(x[3]));
  Py_XSETREF(cur_device, Py_NewRef(x[4]));
  Py_RETURN_NONE;
}

#define FN(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FN("init", f_init),
                                FN("gdn_fwd_varlen", f_fwd),
                                FN("gdn_update", f_upd),
                                FN("attn_norm_rope_cache", f_norm),
                                FN("attn_decode", f_attn),
                                FN("attn_norm_rope_cache_q8", f_norm_q8),
                                FN("kv_cache_read_q8", f_read_q8),
                                FN("attn_decode_q8", f_attn_q8),
                                FN("attn_decode_shared", f_shared),
                                FN("attn_decode_shared_q8", f_shared_q8),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fast(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  return PyModule_Create(&module);
}
