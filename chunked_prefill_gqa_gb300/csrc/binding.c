/*
 * binding.c -- the argument marshalling of the serving-step calls, as a CPython
 * extension: these run once a layer on a handful of rows, where checking seven
 * to fourteen tensors in Python takes three times as long as the launch. Each
 * function here checks its tensors (type, shape, layout, device), collects their
 * addresses and calls the C entry point of the same name; the result is that
 * call's return code. Nothing is computed or kept.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/attn_prefill.h"

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride, *s_cuda_stream, *s_nbytes;
/* torch's own objects, looked up at the first call. */
static PyObject *t_f32, *t_bf16, *t_i32, *t_i64, *f_get_device, *f_raw_stream;

static int setup(void) {
  if (f_raw_stream) return 0;
  PyObject *torch = PyImport_ImportModule("torch"), *c = NULL;
  if (!torch) return -1;
  if ((c = PyObject_GetAttrString(torch, "_C")) && (t_f32 = PyObject_GetAttrString(torch, "float32")) &&
      (t_bf16 = PyObject_GetAttrString(torch, "bfloat16")) && (t_i32 = PyObject_GetAttrString(torch, "int32")) &&
      (t_i64 = PyObject_GetAttrString(torch, "int64")) && (f_get_device = PyObject_GetAttrString(c, "_cuda_getDevice")))
    f_raw_stream = PyObject_GetAttrString(c, "_cuda_getCurrentRawStream");
  Py_XDECREF(c);
  Py_DECREF(torch);
  return f_raw_stream ? 0 : -1;
}

/* What one call has learned: the device its tensors share, -1 before the first. */
typedef struct {
  long dev;
  int failed;
} Call;

#define ANY -1LL

static void *fail(Call *c) {
  c->failed = 1;
  return NULL;
}

/* Reading a property that only a tensor has failed: say so. */
static void *not_a_tensor(Call *c, const char *name) {
  if (PyErr_ExceptionMatches(PyExc_AttributeError)) PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return fail(c);
}

static long long method_int(PyObject *t, PyObject *name) {
  PyObject *v = PyObject_CallMethodNoArgs(t, name);
  if (!v) return -1;
  const long long x = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return x;
}

/*
 * The address of t, a tensor of this dtype and shape (ANY: any extent, which is
 * written back) on the call's device. Contiguous, unless `stride` is given: then
 * [n][heads][64] with the heads of a row packed, and *stride the elements between
 * rows. After a failure every further look returns NULL.
 */
static void *tensor(Call *c, const char *name, PyObject *t, PyObject *dtype, int dims, long long *shape,
                    long long *stride) {
  if (c->failed) return NULL;
  PyObject *got = PyObject_GetAttr(t, s_dtype);
  if (!got) return not_a_tensor(c, name);
  const int same = got == dtype;
  Py_DECREF(got);
  const long long dev = method_int(t, s_get_device);
  if (dev == -1 && PyErr_Occurred()) return not_a_tensor(c, name);
  if (!same || dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a %S CUDA tensor", name, dtype);
    return fail(c);
  }
  if (c->dev < 0) {  /* the first tensor: its device has to be the current one */
    PyObject *v = PyObject_CallNoArgs(f_get_device);
    if (!v) return fail(c);
    c->dev = PyLong_AsLong(v);
    Py_DECREF(v);
  }
  if (dev != c->dev) {
    PyErr_Format(PyExc_ValueError, "%s is on CUDA device %lld, the current device is %ld", name, dev, c->dev);
    return fail(c);
  }
  PyObject *sh = PyObject_GetAttr(t, s_shape);
  if (!sh) return not_a_tensor(c, name);
  int ok = PyTuple_Check(sh) && PyTuple_GET_SIZE(sh) == dims;
  for (int i = 0; ok && i < dims; ++i) {
    const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(sh, i));
    if (shape[i] == ANY) shape[i] = n;
    ok = shape[i] == n;
  }
  if (!ok) {
    PyObject *want = PyTuple_New(dims);
    for (int i = 0; want && i < dims; ++i) PyTuple_SET_ITEM(want, i, PyLong_FromLongLong(shape[i]));
    PyErr_Format(PyExc_ValueError, "%s has shape %S, expected %S", name, sh, want ? want : Py_None);
    Py_XDECREF(want);
    Py_DECREF(sh);
    return fail(c);
  }
  Py_DECREF(sh);
  if (stride) {
    PyObject *st = PyObject_CallMethodNoArgs(t, s_stride);
    if (!st) return not_a_tensor(c, name);
    const int packed = PyTuple_Check(st) && PyTuple_GET_SIZE(st) == 3 &&
                       PyLong_AsLongLong(PyTuple_GET_ITEM(st, 2)) == 1 &&
                       PyLong_AsLongLong(PyTuple_GET_ITEM(st, 1)) == ATTN_D;
    /* with one row the stride has no meaning */
    *stride = packed && shape[0] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(st, 0)) : shape[1] * ATTN_D;
    Py_DECREF(st);
    if (!packed && shape[0] > 0) {
      PyErr_Format(PyExc_ValueError, "%s: the 64 values of a head and the heads of a row must be packed", name);
      return fail(c);
    }
  } else {
    PyObject *v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!v) return not_a_tensor(c, name);
    const int contiguous = v == Py_True;
    Py_DECREF(v);
    if (!contiguous) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return fail(c);
    }
  }
  PyObject *v = PyObject_CallMethodNoArgs(t, s_data_ptr);
  if (!v) return not_a_tensor(c, name);
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!p && PyErr_Occurred()) return fail(c);
  return p;
}

static void *optional(Call *c, const char *name, PyObject *t, PyObject *dtype, int dims, long long *shape) {
  return t == Py_None ? NULL : tensor(c, name, t, dtype, dims, shape, NULL);
}

static int integer(Call *c, const char *name, PyObject *v) {
  if (c->failed) return 0;
  PyObject *i = PyNumber_Index(v);
  int overflow = 0;
  const long x = i ? PyLong_AsLongAndOverflow(i, &overflow) : -1;
  Py_XDECREF(i);
  if (!i) return fail(c), 0;
  if (overflow || x != (int)x) {
    PyErr_Format(PyExc_OverflowError, "%s does not fit an int", name);
    return fail(c), 0;
  }
  return (int)x;
}

/* Sizes that a tensor's extents give: the entry points take ints. */
static int extent(Call *c, const char *name, long long n) {
  if (!c->failed && n != (int)n) {
    PyErr_Format(PyExc_ValueError, "%s has too many elements", name);
    c->failed = 1;
  }
  return (int)n;
}

static cudaStream_t stream_of(Call *c, PyObject *s) {
  PyObject *v = NULL;
  if (c->failed) return NULL;
  if (s == Py_None) {
    PyObject *dev = PyLong_FromLong(c->dev < 0 ? 0 : c->dev);
    v = dev ? PyObject_CallOneArg(f_raw_stream, dev) : NULL;
    Py_XDECREF(dev);
  } else if (PyLong_Check(s)) {
    v = Py_NewRef(s);
  } else {
    v = PyObject_GetAttr(s, s_cuda_stream);
  }
  if (!v) return fail(c);
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  if (!p && PyErr_Occurred()) return fail(c);
  return (cudaStream_t)p;
}

/* q, k and what turns them: shared by the row calls. */
typedef struct {
  void *q, *k, *q_out, *q_weight, *k_weight, *cos_sin, *positions;
  long long q_stride, k_stride;
  int type, n, num_positions;
  PyObject *dtype;
  float eps;
} Rows;

static void rows(Call *c, Rows *r, PyObject *q, PyObject *k, PyObject *positions, PyObject *cos_sin, PyObject *q_out,
                 PyObject *q_weight, PyObject *k_weight, PyObject *eps) {
  memset(r, 0, sizeof(*r));
  PyObject *dtype = PyObject_GetAttr(k, s_dtype);
  if (!dtype) {
    not_a_tensor(c, "k");
    return;
  }
  r->type = dtype == t_f32 ? ATTN_F32 : ATTN_BF16;
  r->dtype = dtype == t_f32 ? t_f32 : t_bf16;
  const int known = dtype == t_f32 || dtype == t_bf16;
  if (!known) {
    PyObject *dev = PyObject_GetAttr(k, s_get_device);
    if (!dev) not_a_tensor(c, "k");
    else PyErr_Format(PyExc_ValueError, "k must be float32 or bfloat16, got %S", dtype);
    Py_XDECREF(dev);
    Py_DECREF(dtype);
    c->failed = 1;
    return;
  }
  Py_DECREF(dtype);
  long long ks[3] = {ANY, ATTN_HKV, ATTN_D};
  r->k = tensor(c, "k", k, r->dtype, 3, ks, &r->k_stride);
  r->n = extent(c, "k", ks[0]);
  long long qs[3] = {ks[0], ATTN_HQ, ATTN_D}, w[1] = {ATTN_D}, tab[2] = {ANY, ATTN_D}, pos[1] = {ks[0]};
  if (q != Py_None) {
    r->q = tensor(c, "q", q, r->dtype, 3, qs, &r->q_stride);
    r->q_out = tensor(c, "qOut", q_out, t_f32, 3, qs, NULL);
  }
  r->q_weight = optional(c, "qWeight", q_weight, t_f32, 1, w);
  r->k_weight = optional(c, "kWeight", k_weight, t_f32, 1, w);
  if (cos_sin != Py_None) {
    r->cos_sin = tensor(c, "cosSin", cos_sin, t_f32, 2, tab, NULL);
    r->num_positions = extent(c, "cosSin", tab[0]);
  }
  r->positions = optional(c, "positions", positions, t_i32, 1, pos);
  if (c->failed) return;
  r->eps = (float)PyFloat_AsDouble(eps);
  if (PyErr_Occurred()) c->failed = 1;
}

/* A paged batch: pages, table, lengths. */
typedef struct {
  void *k_pages, *v_pages, *table, *ctx;
  int B, max_blocks, num_pages;
} Batch;

static void batch(Call *c, Batch *x, int bf16, PyObject *k_pages, PyObject *v_pages, PyObject *table, PyObject *ctx) {
  long long pool[4] = {ANY, ATTN_PAGE, ATTN_HKV, ATTN_D}, len[1] = {ANY};
  PyObject *dtype = bf16 ? t_bf16 : t_f32;
  x->k_pages = tensor(c, "kPages", k_pages, dtype, 4, pool, NULL);
  x->v_pages = tensor(c, "vPages", v_pages, dtype, 4, pool, NULL);
  x->ctx = tensor(c, "contextLens", ctx, t_i32, 1, len, NULL);
  long long tab[2] = {len[0], ANY};
  x->table = tensor(c, "blockTable", table, t_i32, 2, tab, NULL);
  x->B = extent(c, "contextLens", len[0]);
  x->max_blocks = extent(c, "blockTable", tab[1]);
  x->num_pages = extent(c, "kPages", pool[0]);
}

#define CALL(expr)                         \
  int rc;                                  \
  if (c.failed) return NULL;               \
  Py_BEGIN_ALLOW_THREADS rc = (expr);      \
  Py_END_ALLOW_THREADS return PyLong_FromLong(rc)

static PyObject *wrong_count(const char *name) {
  PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", name);
  return NULL;
}

/* q, k, positions, cosSin, qOut, kOut, qWeight, kWeight, eps, pairing, stream */
static PyObject *qk_norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != 11) return wrong_count("qk_norm_rope");
  if (setup()) return NULL;
  Call c = {-1, 0};
  Rows r;
  rows(&c, &r, a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8]);
  if (c.failed) return NULL;
  PyObject *dtype = PyObject_GetAttr(a[5], s_dtype);
  if (!dtype) return not_a_tensor(&c, "kOut");
  const int out = dtype == t_bf16 ? ATTN_BF16 : ATTN_F32;
  Py_DECREF(dtype);
  long long ks[3] = {r.n, ATTN_HKV, ATTN_D};
  void *k_out = tensor(&c, "kOut", a[5], out == ATTN_BF16 ? t_bf16 : t_f32, 3, ks, NULL);
  const int pairing = integer(&c, "pairing", a[9]);
  cudaStream_t st = stream_of(&c, a[10]);
  CALL(attn_qk_norm_rope(r.q, r.k, r.type, r.q_stride, r.k_stride, r.q_weight, r.k_weight, r.eps, r.cos_sin,
                         r.positions, r.num_positions, pairing, r.q_out, k_out, out, r.n, st));
}

/* bf16 pages, k, v, kPages, vPages, blockTable, contextLens, rowStart, cosSin, positions, kWeight, q, qOut, qWeight,
   eps, pairing, stream */
static PyObject *append_paged(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != 17) return wrong_count("append_paged");
  if (setup()) return NULL;
  Call c = {-1, 0};
  const int bf16 = a[0] == Py_True;
  Rows r;
  rows(&c, &r, a[11], a[1], a[9], a[8], a[12], a[13], a[10], a[14]);
  if (c.failed) return NULL;
  long long vs[3] = {r.n, ATTN_HKV, ATTN_D}, v_stride = 0;
  void *v = tensor(&c, "v", a[2], r.dtype, 3, vs, &v_stride);
  Batch x;
  batch(&c, &x, bf16, a[3], a[4], a[5], a[6]);
  long long st1[1] = {(long long)x.B + 1};
  void *starts = tensor(&c, "rowStart", a[7], t_i32, 1, st1, NULL);
  const int pairing = integer(&c, "pairing", a[15]);
  cudaStream_t st = stream_of(&c, a[16]);
  if (bf16) {
    CALL(attn_append_paged_bf16kv(r.q, r.k, v, r.type, r.q_stride, r.k_stride, v_stride, r.q_weight, r.k_weight, r.eps,
                                  r.cos_sin, r.positions, r.num_positions, pairing, r.q_out, x.k_pages, x.v_pages,
                                  x.table, x.ctx, starts, x.B, r.n, x.max_blocks, x.num_pages, st));
  }
  CALL(attn_append_paged(r.q, r.k, v, r.type, r.q_stride, r.k_stride, v_stride, r.q_weight, r.k_weight, r.eps,
                         r.cos_sin, r.positions, r.num_positions, pairing, r.q_out, x.k_pages, x.v_pages, x.table,
                         x.ctx, starts, x.B, r.n, x.max_blocks, x.num_pages, st));
}

/* bf16 pages, q, kPages, vPages, blockTable, contextLens, rowStart, masks, out, max_rows, max_context, num_splits,
   workspace, stream */
static PyObject *tree_paged(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != 14) return wrong_count("tree_paged");
  if (setup()) return NULL;
  Call c = {-1, 0};
  const int bf16 = a[0] == Py_True;
  long long qs[3] = {ANY, ATTN_HQ, ATTN_D};
  void *q = tensor(&c, "q", a[1], t_f32, 3, qs, NULL);
  void *out = tensor(&c, "out", a[8], t_f32, 3, qs, NULL);
  const int rows_n = extent(&c, "q", qs[0]);
  Batch x;
  batch(&c, &x, bf16, a[2], a[3], a[4], a[5]);
  long long st1[1] = {(long long)x.B + 1}, ms[1] = {qs[0]};
  void *starts = tensor(&c, "rowStart", a[6], t_i32, 1, st1, NULL);
  void *masks = optional(&c, "masks", a[7], t_i64, 1, ms);
  const int max_rows = integer(&c, "max_rows", a[9]), max_context = integer(&c, "max_context", a[10]),
            splits = integer(&c, "num_splits", a[11]);
  void *ws = NULL;
  size_t bytes = 0;
  if (a[12] != Py_None && !c.failed) {  /* any type and shape */
    PyObject *dtype = PyObject_GetAttr(a[12], s_dtype), *nb = PyObject_GetAttr(a[12], s_nbytes),
             *sh = PyObject_GetAttr(a[12], s_shape);
    if (!dtype || !nb || !sh || !PyTuple_Check(sh)) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "workspace must be a torch.Tensor");
      not_a_tensor(&c, "workspace");
    } else {
      long long any[8] = {ANY, ANY, ANY, ANY, ANY, ANY, ANY, ANY};
      const int dims = (int)PyTuple_GET_SIZE(sh);
      if (dims > 8) {
        PyErr_SetString(PyExc_ValueError, "workspace has too many dimensions");
        c.failed = 1;
      }
      bytes = PyLong_AsSize_t(nb);
      ws = tensor(&c, "workspace", a[12], dtype, dims, any, NULL);
    }
    Py_XDECREF(dtype);
    Py_XDECREF(nb);
    Py_XDECREF(sh);
  }
  cudaStream_t st = stream_of(&c, a[13]);
  if (bf16) {
    CALL(attn_tree_paged_bf16kv(q, x.k_pages, x.v_pages, x.table, x.ctx, starts, masks, out, x.B, rows_n, max_rows,
                                x.max_blocks, x.num_pages, max_context, splits, ws, bytes, st));
  }
  CALL(attn_tree_paged(q, x.k_pages, x.v_pages, x.table, x.ctx, starts, masks, out, x.B, rows_n, max_rows, x.max_blocks,
                       x.num_pages, max_context, splits, ws, bytes, st));
}

/* bf16 pages, kPages, vPages, blockTable, contextLens, keep, keepCounts, max_rows, stream */
static PyObject *compact_paged(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  if (n != 9) return wrong_count("compact_paged");
  if (setup()) return NULL;
  Call c = {-1, 0};
  const int bf16 = a[0] == Py_True;
  Batch x;
  batch(&c, &x, bf16, a[1], a[2], a[3], a[4]);
  long long ks[2] = {x.B, ANY}, cs[1] = {x.B};
  void *keep = tensor(&c, "keep", a[5], t_i32, 2, ks, NULL);
  void *counts = tensor(&c, "keepCounts", a[6], t_i32, 1, cs, NULL);
  const int max_keep = extent(&c, "keep", ks[1]), max_rows = integer(&c, "max_rows", a[7]);
  cudaStream_t st = stream_of(&c, a[8]);
  if (bf16) {
    CALL(attn_compact_paged_bf16kv(x.k_pages, x.v_pages, x.table, x.ctx, keep, counts, x.B, max_keep, max_rows,
                                   x.max_blocks, x.num_pages, st));
  }
  CALL(attn_compact_paged(x.k_pages, x.v_pages, x.table, x.ctx, keep, counts, x.B, max_keep, max_rows, x.max_blocks,
                          x.num_pages, st));
}

static PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, "attn_qk_norm_rope"},
    {"append_paged", (PyCFunction)(void (*)(void))append_paged, METH_FASTCALL, "attn_append_paged(_bf16kv)"},
    {"tree_paged", (PyCFunction)(void (*)(void))tree_paged, METH_FASTCALL, "attn_tree_paged(_bf16kv)"},
    {"compact_paged", (PyCFunction)(void (*)(void))compact_paged, METH_FASTCALL, "attn_compact_paged(_bf16kv)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "argument marshalling of the serving-step calls",
                                    -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_stride = PyUnicode_InternFromString("stride");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  s_nbytes = PyUnicode_InternFromString("nbytes");
  return s_nbytes ? PyModule_Create(&module) : NULL;
}
