/* CPython entry points of the small-call operators (idx_attn_paged, idx_attn_blocks,
 * idx_store_kv, the same over NVFP4 caches, idx_add_rmsnorm_fp8, idx_norm_rope_store).
 *
 * A decode step's calls take a few microseconds on the GPU, less than ctypes and the
 * checks in Python take on the host (12 us a call of the attention, 6 here).  These
 * functions make the same checks on the tensors' attributes in C and call the library.
 * They handle the ordinary call: positional arguments, contiguous tensors of the right
 * types and shapes on the current device, its current stream.  Anything else (keywords, a given
 * stream, an argument that is wrong) goes to the Python function of the same name, which
 * accepts it or says what is wrong with it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "../../include/idx.h"

static PyObject *s_dtype, *s_shape, *s_is_contiguous, *s_data_ptr, *s_get_device,
    *s_nbytes, *s_stride, *s_element_size;
static PyObject *t_bf16, *t_f32, *t_i32, *t_i64, *t_u8, *t_e4m3; /* torch dtypes */
static PyObject *py_raw_stream, *py_current_device, *py_check;   /* callables */
enum { SLOW_PAGED, SLOW_BLOCKS, SLOW_STORE, SLOW_NORM, SLOW_PAGED4, SLOW_BLOCKS4, SLOW_STORE4, SLOW_ROPE, SLOW_CALLS };
static PyObject *py_slow[SLOW_CALLS];

/* The value of an integer attribute, or of a method without arguments; -1 with no error
 * set where there is none (no quantity here is negative). */
static long long as_int(PyObject* v) {
  long long x = -1;
  if (v) {
    x = PyLong_AsLongLong(v);
    Py_DECREF(v);
  }
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return -1;
  }
  return x;
}
static long long int_attr(PyObject* t, PyObject* name) { return as_int(PyObject_GetAttr(t, name)); }
static long long int_call(PyObject* t, PyObject* name) {
  return as_int(PyObject_CallMethodNoArgs(t, name));
}
static int is_true(PyObject* v) {
  const int yes = v == Py_True;
  if (!v) PyErr_Clear();
  Py_XDECREF(v);
  return yes;
}
static int has_dtype(PyObject* t, PyObject* dtype) {
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (!v) PyErr_Clear();
  const int yes = v == dtype;
  Py_XDECREF(v);
  return yes;
}

/* Integers of a tuple: as many as `n`, which must be its length. */
static int ints_of(PyObject* v, int n, long long* out) {
  int ok = v && PyTuple_Check(v) && PyTuple_GET_SIZE(v) == n;
  if (!v) PyErr_Clear();
  for (int i = 0; ok && i < n; ++i) {
    out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = 0;
    }
  }
  Py_XDECREF(v);
  return ok;
}
static int shape_of(PyObject* t, int n, long long* out) {
  return ints_of(PyObject_GetAttr(t, s_shape), n, out);
}

/* Device pointer of a tensor on device `dev`, contiguous where asked for. */
static int pointer(PyObject* t, int contiguous, long long dev, const void** out) {
  if (dev < 0 || int_call(t, s_get_device) != dev) return 0;
  if (contiguous && !is_true(PyObject_CallMethodNoArgs(t, s_is_contiguous))) return 0;
  PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!v) {
    PyErr_Clear();
    return 0;
  }
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return 1;
}

/* A contiguous tensor of this dtype and shape (n dims). */
static int tensor(PyObject* t, PyObject* dtype, int n, const long long* dims, long long dev,
                  const void** out) {
  long long got[4];
  if (!has_dtype(t, dtype) || !shape_of(t, n, got)) return 0;
  for (int i = 0; i < n; ++i)
    if (got[i] != dims[i]) return 0;
  return pointer(t, 1, dev, out);
}

/* One plane of a cache: payload rows of 128 elements, scale fp32 a row (e4m3), or eight
 * bytes a row (NVFP4). */
static int plane(PyObject* payload, PyObject* scale, int dtype, long long dev,
                 long long* head_pages, const void** p, const void** s) {
  long long dims[2];
  const long long want = dtype == IDX_BF16 ? 256 : dtype == IDX_NVFP4 ? 64 : 128;
  if (!shape_of(payload, 2, dims) || dims[1] * int_call(payload, s_element_size) != want ||
      dims[0] % IDX_PAGE_SIZE != 0 || !pointer(payload, 1, dev, p))
    return 0;
  *head_pages = dims[0] / IDX_PAGE_SIZE;
  *s = NULL;
  if (dtype == IDX_BF16) return scale == Py_None;
  if (dtype == IDX_NVFP4) {
    const long long sdims[2] = {dims[0], IDX_DIM / 16};
    return scale != Py_None && tensor(scale, has_dtype(scale, t_e4m3) ? t_e4m3 : t_u8, 2, sdims, dev, s);
  }
  return scale != Py_None && int_attr(scale, s_nbytes) == dims[0] * 4 && pointer(scale, 1, dev, s);
}

static int kv_dtype_of(PyObject* name) {
  if (!PyUnicode_Check(name)) return -1;
  if (PyUnicode_CompareWithASCIIString(name, "bf16") == 0) return IDX_BF16;
  if (PyUnicode_CompareWithASCIIString(name, "fp8_e4m3") == 0) return IDX_FP8_E4M3;
  return -1;
}

/* The outer scales that end an argument list of n arguments, of which `least` come before
 * them; 0 if the list is of neither length or they are not floats. */
static int outers_of(PyObject* const* a, Py_ssize_t n, Py_ssize_t least, float* k, float* v) {
  *k = *v = 1.f;
  if (n == least) return 1;
  if (n != least + 2 || !PyFloat_CheckExact(a[least]) || !PyFloat_CheckExact(a[least + 1])) return 0;
  *k = (float)PyFloat_AS_DOUBLE(a[least]);
  *v = (float)PyFloat_AS_DOUBLE(a[least + 1]);
  return 1;
}

/* A non-negative C int argument, or -1. */
static int int_arg(PyObject* v) {
  if (!PyLong_CheckExact(v)) return -1;
  const long x = PyLong_AsLong(v);
  if (PyErr_Occurred()) PyErr_Clear();
  return x < 0 || x > 0x7fffffffL ? -1 : (int)x;
}

/* The current device, where the library launches; -1 if torch cannot say. */
static long long device_here(void) { return as_int(PyObject_CallNoArgs(py_current_device)); }

/* Its current stream. */
static int stream_of(long long dev, void** out) {
  PyObject* d = PyLong_FromLongLong(dev);
  PyObject* v = d ? PyObject_CallOneArg(py_raw_stream, d) : NULL;
  Py_XDECREF(d);
  if (!v) {
    PyErr_Clear();
    return 0;
  }
  *out = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return 1;
}

static PyObject* slow(int which, PyObject* const* args, Py_ssize_t n, PyObject* kw) {
  return PyObject_Vectorcall(py_slow[which], args, (size_t)n, kw);
}

static PyObject* done(int rc, const char* what) {
  if (rc == IDX_OK) Py_RETURN_NONE;
  return PyObject_CallFunction(py_check, "is", rc, what);
}

/* (q, k_payload, k_scale, v_payload, v_scale, [kv_dtype,] page_table, slot_ids, row_lens,
 *  [block_ids, lists,] kv_heads, sm_scale, out, out_lse, workspace[, k_outer, v_outer]): the
 * dtype for bf16 and e4m3 caches, the outer scales for NVFP4 ones (fp4). */
static PyObject* attn(int blocks, int fp4, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  const int which = fp4 ? (blocks ? SLOW_BLOCKS4 : SLOW_PAGED4) : blocks ? SLOW_BLOCKS : SLOW_PAGED;
  const Py_ssize_t least = (blocks ? 16 : 14) - fp4;
  float ko = 1.f, vo = 1.f;
  if (kw || (fp4 ? !outers_of(a, n, least, &ko, &vo) : n != least)) return slow(which, a, n, kw);
  PyObject* const* t = a + 6 - fp4;            /* page_table onwards */
  PyObject* const* b = t + (blocks ? 5 : 3);   /* kv_heads onwards */
  const void *q, *kp, *ks, *vp, *vs, *table, *slots, *lens, *ids = NULL, *out, *lse = NULL, *ws;
  long long qs[4], tb[2], ib[3] = {0, 0, 0}, kpages, vpages;
  const long long dev = device_here();
  void* stream;
  const int dtype = fp4 ? IDX_NVFP4 : kv_dtype_of(a[5]), kv_heads = int_arg(b[0]);
  const int lists = blocks ? int_arg(t[4]) : 1;
  const double scale = PyFloat_CheckExact(b[1]) ? PyFloat_AS_DOUBLE(b[1]) : 0.0;
  if (dtype < 0 || kv_heads < 1 || lists < 1 || !(scale > 0) || !shape_of(a[0], 4, qs) ||
      qs[3] != IDX_DIM || qs[0] > IDX_MAX_REQUESTS || qs[1] > IDX_MAX_ROWS_PER_REQUEST ||
      qs[2] > IDX_MAX_ROWS_PER_REQUEST || !tensor(a[0], t_bf16, 4, qs, dev, &q) ||
      !plane(a[1], a[2], dtype, dev, &kpages, &kp, &ks) ||
      !plane(a[3], a[4], dtype, dev, &vpages, &vp, &vs) ||
      kpages != vpages || kpages % kv_heads != 0 || !shape_of(t[0], 2, tb) || tb[0] > 0x7fffffffLL ||
      tb[1] > 65536 || !tensor(t[0], t_i32, 2, tb, dev, &table) ||
      !tensor(t[1], t_i32, 1, qs, dev, &slots) || !tensor(t[2], t_i32, 2, qs, dev, &lens))
    return slow(which, a, n, kw);
  if (blocks && (!shape_of(t[3], 3, ib) || ib[0] != qs[0] || ib[1] != qs[1] * lists ||
                 ib[2] > IDX_MAX_TOPK || !tensor(t[3], t_i32, 3, ib, dev, &ids)))
    return slow(which, a, n, kw);
  if (!tensor(b[2], t_bf16, 4, qs, dev, &out) ||
      (b[3] != Py_None && !tensor(b[3], t_f32, 3, qs, dev, &lse)) || !pointer(b[4], 1, dev, &ws) ||
      !stream_of(dev, &stream))
    return slow(which, a, n, kw);
  const long long ws_bytes = int_attr(b[4], s_nbytes);
  if (ws_bytes < 0) return slow(which, a, n, kw);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  if (fp4 && blocks)
    rc = idx_attn_blocks_nvfp4(q, kp, ks, vp, vs, kpages / kv_heads, kv_heads, table, (int)tb[0],
                               (int)tb[1], slots, lens, ids, lists, (int)ib[2], (int)qs[0], (int)qs[1],
                               (int)qs[2], (float)scale, ko, vo, (void*)out, (float*)lse, (void*)ws,
                               (size_t)ws_bytes, stream);
  else if (fp4)
    rc = idx_attn_paged_nvfp4(q, kp, ks, vp, vs, kpages / kv_heads, kv_heads, table, (int)tb[0],
                              (int)tb[1], slots, lens, (int)qs[0], (int)qs[1], (int)qs[2], (float)scale,
                              ko, vo, (void*)out, (float*)lse, (void*)ws, (size_t)ws_bytes, stream);
  else if (blocks)
    rc = idx_attn_blocks(q, kp, ks, vp, vs, dtype, kpages / kv_heads, kv_heads, table, (int)tb[0],
                         (int)tb[1], slots, lens, ids, lists, (int)ib[2], (int)qs[0], (int)qs[1],
                         (int)qs[2], (float)scale, (void*)out, (float*)lse, (void*)ws,
                         (size_t)ws_bytes, stream);
  else
    rc = idx_attn_paged(q, kp, ks, vp, vs, dtype, kpages / kv_heads, kv_heads, table, (int)tb[0],
                        (int)tb[1], slots, lens, (int)qs[0], (int)qs[1], (int)qs[2], (float)scale,
                        (void*)out, (float*)lse, (void*)ws, (size_t)ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return done(rc, fp4 ? (blocks ? "idx_attn_blocks_nvfp4" : "idx_attn_paged_nvfp4")
                      : blocks ? "idx_attn_blocks" : "idx_attn_paged");
}
static PyObject* py_attn_paged(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return attn(0, 0, a, n, kw);
}
static PyObject* py_attn_blocks(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return attn(1, 0, a, n, kw);
}
static PyObject* py_attn_paged4(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return attn(0, 1, a, n, kw);
}
static PyObject* py_attn_blocks4(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return attn(1, 1, a, n, kw);
}

/* New keys or values [tokens, heads, 128], tokens any stride apart. */
static int source(PyObject* t, long long tokens, int heads, long long dev, const void** p,
                  long long* stride) {
  long long dims[3], st[3];
  if (!has_dtype(t, t_bf16) || !shape_of(t, 3, dims) || dims[0] != tokens || dims[1] != heads ||
      dims[2] != IDX_DIM || !pointer(t, 0, dev, p) ||
      !ints_of(PyObject_CallMethodNoArgs(t, s_stride), 3, st) || st[2] != 1 ||
      (heads > 1 && st[1] != IDX_DIM))
    return 0;
  *stride = tokens > 1 ? st[0] : (long long)heads * IDX_DIM;
  return 1;
}

static int fill_pool(idx_pool* p, PyObject* payload, PyObject* scale, int dtype, long long dev) {
  const void *pp, *ps;
  long long pages;
  if (!plane(payload, scale, dtype, dev, &pages, &pp, &ps)) return 0;
  p->dtype = dtype;
  p->page_size = IDX_PAGE_SIZE;
  p->dim = IDX_DIM;
  p->reserved = 0;
  p->num_pages = pages;
  p->payload = (void*)pp;
  p->scale = (void*)ps;
  p->payload_row_bytes = dtype == IDX_BF16 ? 256 : dtype == IDX_NVFP4 ? 64 : 128;
  p->scale_row_bytes = dtype == IDX_BF16 ? 0 : dtype == IDX_NVFP4 ? 8 : 4;
  return 1;
}

/* (k_src, v_src, slot_mapping, k_payload, k_scale, v_payload, v_scale, kv_dtype, kv_heads), or
 * (.., v_scale, kv_heads[, k_outer, v_outer]) for NVFP4 */
static PyObject* store(int fp4, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  const int which = fp4 ? SLOW_STORE4 : SLOW_STORE;
  float ko = 1.f, vo = 1.f;
  if (kw || (fp4 ? !outers_of(a, n, 8, &ko, &vo) : n != 9)) return slow(which, a, n, kw);
  const int dtype = fp4 ? IDX_NVFP4 : kv_dtype_of(a[7]), heads = int_arg(a[8 - fp4]), values = a[1] != Py_None;
  const void *k, *v = NULL, *slots;
  const long long dev = device_here();
  long long tokens, ks, vs = 0;
  idx_pool kp, vp;
  void* stream;
  if (dtype < 0 || heads < 1 || (a[5] != Py_None) != values || !shape_of(a[2], 1, &tokens) ||
      !tensor(a[2], t_i64, 1, &tokens, dev, &slots) || !source(a[0], tokens, heads, dev, &k, &ks) ||
      !fill_pool(&kp, a[3], a[4], dtype, dev) ||
      (values && (!source(a[1], tokens, heads, dev, &v, &vs) || !fill_pool(&vp, a[5], a[6], dtype, dev))) ||
      (!values && a[6] != Py_None) || !stream_of(dev, &stream))
    return slow(which, a, n, kw);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  if (fp4)
    rc = idx_store_kv_nvfp4(k, v, ks, vs, (const int64_t*)slots, tokens, heads, &kp, values ? &vp : NULL,
                            ko, vo, stream);
  else
    rc = idx_store_kv(k, v, ks, vs, (const int64_t*)slots, tokens, heads, &kp, values ? &vp : NULL, stream);
  Py_END_ALLOW_THREADS
  return done(rc, fp4 ? "idx_store_kv_nvfp4" : "idx_store_kv");
}
static PyObject* py_store_kv(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return store(0, a, n, kw);
}
static PyObject* py_store_kv4(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  return store(1, a, n, kw);
}

/* (q, k, v, q_weight, k_weight, eps, table, positions, pair_axis, interleaved, slot_mapping, out_q,
 *  out_q_scale, k_payload, k_scale, v_payload, v_scale, kv_dtype, kv_heads[, k_outer, v_outer]) */
static PyObject* py_norm_rope_store(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  float ko, vo;
  if (kw || !outers_of(a, n, 19, &ko, &vo)) return slow(SLOW_ROPE, a, n, kw);
  const int values = a[2] != Py_None, queries = a[0] != Py_None, turned = a[6] != Py_None;
  int dtype = kv_dtype_of(a[17]);
  if (dtype < 0 && PyUnicode_Check(a[17]) && PyUnicode_CompareWithASCIIString(a[17], "nvfp4") == 0) dtype = IDX_NVFP4;
  const int heads = int_arg(a[18]);
  const void *q = NULL, *k, *v = NULL, *qw = NULL, *kwt = NULL, *slots, *out = NULL, *outs = NULL;
  const long long dev = device_here(), dim = IDX_DIM;
  long long tokens, qd[3] = {0, 0, 0}, qs = 0, ks, vs = 0;
  idx_pool kp, vp;
  idx_rope rope;
  void* stream;
  if (dtype < 0 || heads < 1 || (a[15] != Py_None) != values || (a[11] != Py_None) != queries ||
      (!queries && a[12] != Py_None) || (!values && a[16] != Py_None) || !PyFloat_CheckExact(a[5]) ||
      !PyBool_Check(a[9]) || !shape_of(a[10], 1, &tokens) ||
      !tensor(a[10], t_i64, 1, &tokens, dev, &slots) || !source(a[1], tokens, heads, dev, &k, &ks) ||
      !fill_pool(&kp, a[13], a[14], dtype, dev) ||
      (values && (!source(a[2], tokens, heads, dev, &v, &vs) || !fill_pool(&vp, a[15], a[16], dtype, dev))) ||
      (a[3] != Py_None && !tensor(a[3], t_bf16, 1, &dim, dev, &qw)) ||
      (a[4] != Py_None && !tensor(a[4], t_bf16, 1, &dim, dev, &kwt)))
    return slow(SLOW_ROPE, a, n, kw);
  if (queries) {
    PyObject* kind = a[12] == Py_None ? t_bf16 : has_dtype(a[11], t_e4m3) ? t_e4m3 : t_u8;
    if (!shape_of(a[0], 3, qd) || qd[1] < 1 || qd[1] > IDX_MAX_ROWS_PER_REQUEST ||
        !source(a[0], tokens, (int)qd[1], dev, &q, &qs) || !tensor(a[11], kind, 3, qd, dev, &out) ||
        (a[12] != Py_None && !tensor(a[12], t_f32, 2, qd, dev, &outs)))
      return slow(SLOW_ROPE, a, n, kw);
  }
  if (turned) {
    long long tb[2], pd[2] = {1, tokens};
    const void *table, *pos;
    char* by = NULL;
    Py_ssize_t nby = 0;
    if (a[8] != Py_None && (!PyBytes_CheckExact(a[8]) || PyBytes_AsStringAndSize(a[8], &by, &nby) < 0 || nby < 1))
      return slow(SLOW_ROPE, a, n, kw);
    const int flat = shape_of(a[7], 1, pd + 1);
    if (!shape_of(a[6], 2, tb) || tb[1] > IDX_DIM || !tensor(a[6], t_f32, 2, tb, dev, &table) ||
        (!flat && !shape_of(a[7], 2, pd)) || pd[1] != tokens || pd[0] > IDX_MAX_ROPE_AXES ||
        !tensor(a[7], t_i32, flat ? 1 : 2, flat ? pd + 1 : pd, dev, &pos) ||
        ((pd[0] > 1 || by) && nby != tb[1] / 2))
      return slow(SLOW_ROPE, a, n, kw);
    rope = (idx_rope){.table = table, .num_positions = tb[0], .positions = pos, .axes = (int32_t)pd[0],
                      .rotary_dim = (int32_t)tb[1], .interleaved = a[9] == Py_True};
    if (by) memcpy(rope.pair_axis, by, (size_t)nby);
  } else if (a[7] != Py_None || a[8] != Py_None) {
    return slow(SLOW_ROPE, a, n, kw);
  }
  if (!stream_of(dev, &stream)) return slow(SLOW_ROPE, a, n, kw);
  const float eps = (float)PyFloat_AS_DOUBLE(a[5]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = idx_norm_rope_store(q, qs, (int)qd[1], k, ks, v, vs, heads, qw, kwt, eps, turned ? &rope : NULL,
                           (const int64_t*)slots, tokens, (void*)out, (float*)outs, &kp,
                           values ? &vp : NULL, ko, vo, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "idx_norm_rope_store");
}

/* Rows of a bf16 matrix, any stride apart. */
static int rows_2d(PyObject* t, const long long* dims, long long dev, const void** p,
                   long long* stride) {
  long long got[2], st[2];
  if (!has_dtype(t, t_bf16) || !shape_of(t, 2, got) || got[0] != dims[0] || got[1] != dims[1] ||
      !pointer(t, 0, dev, p) || !ints_of(PyObject_CallMethodNoArgs(t, s_stride), 2, st) ||
      (dims[1] > 1 && st[1] != 1))
    return 0;
  *stride = dims[0] > 1 ? st[0] : dims[1];
  return 1;
}

/* (x, residual, weight, eps, group, out, out_scale[, out_residual]) */
static PyObject* py_add_rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n, PyObject* kw) {
  (void)self;
  if (kw || (n != 7 && n != 8)) return slow(SLOW_NORM, a, n, kw);
  const void *x, *r = NULL, *w, *out, *scale, *new_r = NULL;
  const long long dev = device_here();
  long long dims[2], xs, rs = 0;
  void* stream;
  const int group = int_arg(a[4]);
  if (group < 0 || !PyFloat_CheckExact(a[3]) || !shape_of(a[0], 2, dims) ||
      dims[1] > IDX_MAX_NORM_DIM || !rows_2d(a[0], dims, dev, &x, &xs) ||
      (a[1] != Py_None && !rows_2d(a[1], dims, dev, &r, &rs)) ||
      !tensor(a[2], t_bf16, 1, dims + 1, dev, &w) ||
      !tensor(a[5], has_dtype(a[5], t_e4m3) ? t_e4m3 : t_u8, 2, dims, dev, &out))
    return slow(SLOW_NORM, a, n, kw);
  const long long groups = group > 0 ? (dims[1] + group - 1) / group : 1;
  if (!has_dtype(a[6], t_f32) || int_attr(a[6], s_nbytes) != 4 * dims[0] * groups ||
      !pointer(a[6], 1, dev, &scale) ||
      (n == 8 && a[7] != Py_None && !tensor(a[7], t_bf16, 2, dims, dev, &new_r)) ||
      !stream_of(dev, &stream))
    return slow(SLOW_NORM, a, n, kw);
  const float eps = (float)PyFloat_AS_DOUBLE(a[3]);
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = idx_add_rmsnorm_fp8(x, xs, r, rs, w, dims[0], (int)dims[1], group, eps, (void*)out,
                           (float*)scale, (void*)new_r, stream);
  Py_END_ALLOW_THREADS
  return done(rc, "idx_add_rmsnorm_fp8");
}

/* bind(dtypes, raw_stream, current_device, check, slow functions): the Python objects used above. */
static PyObject* py_bind(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *d[6], *stream, *device, *check, *f;
  if (!PyArg_ParseTuple(args, "(OOOOOO)OOOO!", &d[0], &d[1], &d[2], &d[3], &d[4], &d[5], &stream,
                        &device, &check, &PyTuple_Type, &f))
    return NULL;
  if (PyTuple_GET_SIZE(f) != SLOW_CALLS) {
    PyErr_Format(PyExc_TypeError, "bind takes %d functions", (int)SLOW_CALLS);
    return NULL;
  }
  PyObject** to[6] = {&t_bf16, &t_f32, &t_i32, &t_i64, &t_u8, &t_e4m3};
  for (int i = 0; i < 6; ++i) Py_XSETREF(*to[i], Py_NewRef(d[i]));
  Py_XSETREF(py_raw_stream, Py_NewRef(stream));
  Py_XSETREF(py_current_device, Py_NewRef(device));
  Py_XSETREF(py_check, Py_NewRef(check));
  for (int i = 0; i < SLOW_CALLS; ++i) Py_XSETREF(py_slow[i], Py_NewRef(PyTuple_GET_ITEM(f, i)));
  Py_RETURN_NONE;
}

#define FAST(f) (PyCFunction)(void (*)(void))(f), METH_FASTCALL | METH_KEYWORDS
static PyMethodDef methods[] = {
    {"bind", py_bind, METH_VARARGS, "Hand over torch's dtypes, its stream and device calls and the Python functions."},
    {"idx_attn_paged", FAST(py_attn_paged), "Attention over the whole paged cache (see _lib.idx_attn_paged)."},
    {"idx_attn_blocks", FAST(py_attn_blocks), "Attention over block lists (see _lib.idx_attn_blocks)."},
    {"idx_store_kv", FAST(py_store_kv), "Store of new keys and values (see _lib.idx_store_kv)."},
    {"idx_add_rmsnorm_fp8", FAST(py_add_rmsnorm), "Residual, norm, e4m3 (see _lib.idx_add_rmsnorm_fp8)."},
    {"idx_attn_paged_nvfp4", FAST(py_attn_paged4), "The same over an NVFP4 cache (see _lib.idx_attn_paged_nvfp4)."},
    {"idx_attn_blocks_nvfp4", FAST(py_attn_blocks4), "The same over an NVFP4 cache (see _lib.idx_attn_blocks_nvfp4)."},
    {"idx_store_kv_nvfp4", FAST(py_store_kv4), "Store into an NVFP4 cache (see _lib.idx_store_kv_nvfp4)."},
    {"idx_norm_rope_store", FAST(py_norm_rope_store), "Norm, rotation and store (see _lib.idx_norm_rope_store)."},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  const struct { PyObject** to; const char* name; } names[] = {
      {&s_dtype, "dtype"}, {&s_shape, "shape"},
      {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"}, {&s_get_device, "get_device"},
      {&s_nbytes, "nbytes"}, {&s_stride, "stride"}, {&s_element_size, "element_size"}};
  for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
  return PyModule_Create(&module);
}
