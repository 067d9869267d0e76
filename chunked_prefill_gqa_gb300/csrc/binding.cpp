// binding.cpp -- the argument marshalling of the serving-step calls, as a CPython
// extension: these run once a layer on a handful of rows, where looking at seven to
// fourteen tensors in Python takes longer than the launch. Each function here checks
// its tensors (type, shape, layout, device), collects their addresses and calls the
// C entry point of the same name; the result is that call's return code. Nothing is
// computed or kept. (Norm and
// rotation of 7 rows, the host's time for a call: 2.3 us; 4.9 with the tensors looked at
// through their Python methods, 9 in Python.)
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "../../include/attn_prefill.h"

namespace {

// What one call has learned: the device its tensors share, -1 before the first.
struct Call {
  int dev = -1;
  bool failed = false;
};

constexpr long long kAny = -1;
constexpr at::ScalarType kF32 = at::kFloat, kBF16 = at::kBFloat16, kI32 = at::kInt, kI64 = at::kLong;

const char* name_of(at::ScalarType t) {
  return t == kF32 ? "float32" : t == kBF16 ? "bfloat16" : t == kI32 ? "int32" : t == kI64 ? "int64" : at::toString(t);
}

const at::Tensor* unpack(Call* c, const char* name, PyObject* t) {
  if (c->failed) return nullptr;
  if (!THPVariable_Check(t)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    c->failed = true;
    return nullptr;
  }
  return &THPVariable_Unpack(t);
}

template <typename... A>
void* fail(Call* c, const char* format, A... args) {
  PyErr_Format(PyExc_ValueError, format, args...);
  c->failed = true;
  return nullptr;
}

std::string text(int dims, const long long* shape) {
  std::string s = "(";
  for (int i = 0; i < dims; ++i) s += (i ? ", " : "") + (shape[i] == kAny ? std::string("any") : std::to_string(shape[i]));
  return s + ")";
}

// The address of t, a tensor of this dtype and shape (kAny: any extent, which is
// written back) on the call's device. Contiguous, unless `stride` is given: then
// [n][heads][64] with the heads of a row packed, and *stride the elements between
// rows. After a failure every further look returns nullptr.
void* tensor(Call* c, const char* name, PyObject* t, at::ScalarType dtype, int dims, long long* shape,
             long long* stride = nullptr) {
  const at::Tensor* x = unpack(c, name, t);
  if (!x) return nullptr;
  if (x->scalar_type() != dtype || !x->is_cuda()) return fail(c, "%s must be a %s CUDA tensor", name, name_of(dtype));
  const int dev = x->get_device();
  if (c->dev < 0) c->dev = c10::cuda::current_device();  // the first tensor's has to be the current one
  if (dev != c->dev) return fail(c, "%s is on CUDA device %d, the current device is %d", name, dev, c->dev);
  const at::IntArrayRef sizes = x->sizes();
  bool same = (int)sizes.size() == dims;
  for (int i = 0; same && i < dims; ++i) {
    if (shape[i] == kAny) shape[i] = sizes[i];
    same = shape[i] == sizes[i];
  }
  if (!same) {
    long long got[8];
    const int n = (int)sizes.size() < 8 ? (int)sizes.size() : 8;
    for (int i = 0; i < n; ++i) got[i] = sizes[i];
    return fail(c, "%s has shape %s, expected %s", name, text(n, got).c_str(), text(dims, shape).c_str());
  }
  if (stride) {
    const at::IntArrayRef strides = x->strides();
    const bool packed = strides[2] == 1 && strides[1] == ATTN_D;
    // with one row the stride has no meaning
    *stride = packed && shape[0] > 1 ? strides[0] : shape[1] * ATTN_D;
    if (!packed && shape[0] > 0)
      return fail(c, "%s: the 64 values of a head and the heads of a row must be packed", name);
  } else if (!x->is_contiguous()) {
    return fail(c, "%s must be contiguous", name);
  }
  return x->data_ptr();
}

void* optional(Call* c, const char* name, PyObject* t, at::ScalarType dtype, int dims, long long* shape) {
  return t == Py_None ? nullptr : tensor(c, name, t, dtype, dims, shape);
}

int integer(Call* c, const char* name, PyObject* v) {
  if (c->failed) return 0;
  PyObject* i = PyNumber_Index(v);
  int overflow = 0;
  const long x = i ? PyLong_AsLongAndOverflow(i, &overflow) : -1;
  Py_XDECREF(i);
  if (!i || overflow || x != (int)x) {
    if (i) PyErr_Format(PyExc_OverflowError, "%s does not fit an int", name);
    c->failed = true;
    return 0;
  }
  return (int)x;
}

// Sizes that a tensor's extents give: the entry points take ints.
int extent(Call* c, const char* name, long long n) {
  if (!c->failed && n != (int)n) fail(c, "%s has too many elements", name);
  return (int)n;
}

cudaStream_t stream_of(Call* c, PyObject* s) {
  if (c->failed) return nullptr;
  if (s == Py_None) return c10::cuda::getCurrentCUDAStream(c->dev < 0 ? 0 : c->dev).stream();
  PyObject* v = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
  void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
  Py_XDECREF(v);
  if (!v || (!p && PyErr_Occurred())) c->failed = true;
  return (cudaStream_t)p;
}

// q, k and what turns them: shared by the row calls.
struct Rows {
  void *q = nullptr, *k = nullptr, *q_out = nullptr, *q_weight = nullptr, *k_weight = nullptr, *cos_sin = nullptr,
       *positions = nullptr;
  long long q_stride = 0, k_stride = 0;
  int type = 0, n = 0, num_positions = 0;
  at::ScalarType dtype = kF32;
  float eps = 0.f;
};

void rows(Call* c, Rows* r, PyObject* q, PyObject* k, PyObject* positions, PyObject* cos_sin, PyObject* q_out,
          PyObject* q_weight, PyObject* k_weight, PyObject* eps) {
  const at::Tensor* x = unpack(c, "k", k);
  if (!x) return;
  r->dtype = x->scalar_type();
  r->type = r->dtype == kF32 ? ATTN_F32 : ATTN_BF16;
  if (r->dtype != kF32 && r->dtype != kBF16) {
    fail(c, "k must be float32 or bfloat16, got %s", name_of(r->dtype));
    return;
  }
  long long ks[3] = {kAny, ATTN_HKV, ATTN_D};
  r->k = tensor(c, "k", k, r->dtype, 3, ks, &r->k_stride);
  r->n = extent(c, "k", ks[0]);
  long long qs[3] = {ks[0], ATTN_HQ, ATTN_D}, w[1] = {ATTN_D}, tab[2] = {kAny, ATTN_D}, pos[1] = {ks[0]};
  if (q != Py_None) {
    r->q = tensor(c, "q", q, r->dtype, 3, qs, &r->q_stride);
    r->q_out = tensor(c, "qOut", q_out, kF32, 3, qs);
  }
  r->q_weight = optional(c, "qWeight", q_weight, kF32, 1, w);
  r->k_weight = optional(c, "kWeight", k_weight, kF32, 1, w);
  if (cos_sin != Py_None) {
    r->cos_sin = tensor(c, "cosSin", cos_sin, kF32, 2, tab);
    r->num_positions = extent(c, "cosSin", tab[0]);
  }
  r->positions = optional(c, "positions", positions, kI32, 1, pos);
  if (c->failed) return;
  r->eps = (float)PyFloat_AsDouble(eps);
  if (PyErr_Occurred()) c->failed = true;
}

// A row's positions on several axes, and the axis of each frequency.
struct Axes {
  const int* positions = nullptr;
  long long stride = 0;
  int count = 0, of[ATTN_D / 2] = {};
};

void axes_of(Call* c, Axes* x, long long n, PyObject* positions, PyObject* axes) {
  const at::Tensor* p = unpack(c, "positions", positions);
  if (!p) return;
  if (p->scalar_type() != kI32 || !p->is_cuda()) {
    fail(c, "positions must be a %s CUDA tensor", name_of(kI32));
    return;
  }
  if (c->dev < 0) c->dev = c10::cuda::current_device();
  if (p->get_device() != c->dev) {
    fail(c, "positions is on CUDA device %d, the current device is %d", (int)p->get_device(), c->dev);
    return;
  }
  if (p->dim() != 2 || p->size(1) != n) {
    fail(c, "positions must be [axes][%lld]", n);
    return;
  }
  if (n > 1 && p->stride(1) != 1) {
    fail(c, "positions: those of an axis must be packed");
    return;
  }
  x->positions = (const int*)p->data_ptr();
  x->count = extent(c, "positions", p->size(0));
  x->stride = x->count > 1 ? p->stride(0) : 0;
  PyObject* seq = PySequence_Fast(axes, "axes must be a sequence of 32 ints");
  if (!seq) {
    c->failed = true;
    return;
  }
  if (PySequence_Fast_GET_SIZE(seq) != ATTN_D / 2) fail(c, "axes must hold %d axes", ATTN_D / 2);
  for (int i = 0; i < ATTN_D / 2 && !c->failed; ++i) x->of[i] = integer(c, "axes", PySequence_Fast_GET_ITEM(seq, i));
  Py_DECREF(seq);
}

// Any tensor of the call's device, as bytes; None: none.
void* workspace_of(Call* c, PyObject* t, size_t* bytes) {
  *bytes = 0;
  if (t == Py_None) return nullptr;
  const at::Tensor* w = unpack(c, "workspace", t);
  if (!w) return nullptr;
  long long any[8] = {kAny, kAny, kAny, kAny, kAny, kAny, kAny, kAny};
  if (w->dim() > 8) return fail(c, "workspace has too many dimensions");
  void* p = tensor(c, "workspace", t, w->scalar_type(), (int)w->dim(), any);
  if (!c->failed) *bytes = w->nbytes();
  return p;
}

float real(Call* c, PyObject* v) {
  if (c->failed) return 0.f;
  const double x = PyFloat_AsDouble(v);
  if (PyErr_Occurred()) c->failed = true;
  return (float)x;
}

// A paged batch: pages, table, lengths.
struct Batch {
  void *k_pages, *v_pages, *table, *ctx;
  float* weights;
  int B, max_blocks, num_pages;
};

// v_pages or weights nullptr: the call has none.
void batch(Call* c, Batch* x, bool bf16, PyObject* k_pages, PyObject* v_pages, PyObject* table, PyObject* ctx,
           PyObject* weights = nullptr) {
  long long pool[4] = {kAny, ATTN_PAGE, ATTN_HKV, ATTN_D}, len[1] = {kAny};
  const at::ScalarType dtype = bf16 ? kBF16 : kF32;
  x->k_pages = tensor(c, "kPages", k_pages, dtype, 4, pool);
  x->v_pages = v_pages ? tensor(c, "vPages", v_pages, dtype, 4, pool) : nullptr;
  long long by_page[3] = {pool[0], ATTN_HKV, ATTN_PAGE};
  x->weights = weights ? (float*)tensor(c, "weights", weights, kF32, 3, by_page) : nullptr;
  x->ctx = tensor(c, "contextLens", ctx, kI32, 1, len);
  long long tab[2] = {len[0], kAny};
  x->table = tensor(c, "blockTable", table, kI32, 2, tab);
  x->B = extent(c, "contextLens", len[0]);
  x->max_blocks = extent(c, "blockTable", tab[1]);
  x->num_pages = extent(c, "kPages", pool[0]);
}

// One entry: the number of arguments, and no C++ exception past it. `body` returns
// the library's code through call().
template <typename F>
PyObject* entry(const char* name, Py_ssize_t got, Py_ssize_t want, F body) {
  if (got != want) return PyErr_Format(PyExc_TypeError, "%s: wrong number of arguments", name);
  try {
    return body();
  } catch (const std::exception& e) {
    return PyErr_Format(PyExc_RuntimeError, "%s: %s", name, e.what());
  }
}
template <typename F>
PyObject* call(const Call& c, F f) {
  if (c.failed) return nullptr;
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
}

// q, k, positions, cosSin, qOut, kOut, qWeight, kWeight, eps, pairing, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("qk_norm_rope", n, 11, [&]() -> PyObject* {
    Call c;
    Rows r;
    rows(&c, &r, a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8]);
    const at::Tensor* ko = unpack(&c, "kOut", a[5]);
    if (!ko) return nullptr;
    const bool bf16 = ko->scalar_type() == kBF16;
    long long ks[3] = {r.n, ATTN_HKV, ATTN_D};
    void* k_out = tensor(&c, "kOut", a[5], bf16 ? kBF16 : kF32, 3, ks);
    const int pairing = integer(&c, "pairing", a[9]);
    const cudaStream_t st = stream_of(&c, a[10]);
    return call(c, [&] {
      return attn_qk_norm_rope(r.q, r.k, r.type, r.q_stride, r.k_stride, (const float*)r.q_weight,
                               (const float*)r.k_weight, r.eps, (const float*)r.cos_sin, (const int*)r.positions,
                               r.num_positions, pairing, (float*)r.q_out, k_out, bf16 ? ATTN_BF16 : ATTN_F32, r.n, st);
    });
  });
}

// bf16 pages, k, v, kPages, vPages, blockTable, contextLens, rowStart, cosSin, positions, kWeight, q, qOut, qWeight,
// eps, pairing, stream
PyObject* append_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("append_paged", n, 17, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Rows r;
    rows(&c, &r, a[11], a[1], a[9], a[8], a[12], a[13], a[10], a[14]);
    long long vs[3] = {r.n, ATTN_HKV, ATTN_D}, v_stride = 0;
    void* v = tensor(&c, "v", a[2], r.dtype, 3, vs, &v_stride);
    Batch x;
    batch(&c, &x, bf16, a[3], a[4], a[5], a[6]);
    long long st1[1] = {(long long)x.B + 1};
    const int* starts = (const int*)tensor(&c, "rowStart", a[7], kI32, 1, st1);
    const int pairing = integer(&c, "pairing", a[15]);
    const cudaStream_t st = stream_of(&c, a[16]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(r.q, r.k, v, r.type, r.q_stride, r.k_stride, v_stride, (const float*)r.q_weight,
                  (const float*)r.k_weight, r.eps, (const float*)r.cos_sin, (const int*)r.positions, r.num_positions,
                  pairing, (float*)r.q_out, k_pages, v_pages, (const int*)x.table, (const int*)x.ctx, starts, x.B, r.n,
                  x.max_blocks, x.num_pages, st);
      };
      return bf16 ? go(attn_append_paged_bf16kv, (uint16_t*)x.k_pages, (uint16_t*)x.v_pages)
                  : go(attn_append_paged, (float*)x.k_pages, (float*)x.v_pages);
    });
  });
}

// q, k, positions, axes, cosSin, qOut, kOut, qWeight, kWeight, eps, pairing, stream
PyObject* qk_norm_rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("qk_norm_rope_axes", n, 12, [&]() -> PyObject* {
    Call c;
    Rows r;
    rows(&c, &r, a[0], a[1], Py_None, a[4], a[5], a[7], a[8], a[9]);
    Axes x;
    axes_of(&c, &x, r.n, a[2], a[3]);
    const at::Tensor* ko = unpack(&c, "kOut", a[6]);
    if (!ko) return nullptr;
    const bool bf16 = ko->scalar_type() == kBF16;
    long long ks[3] = {r.n, ATTN_HKV, ATTN_D};
    void* k_out = tensor(&c, "kOut", a[6], bf16 ? kBF16 : kF32, 3, ks);
    const int pairing = integer(&c, "pairing", a[10]);
    const cudaStream_t st = stream_of(&c, a[11]);
    return call(c, [&] {
      return attn_qk_norm_rope_axes(r.q, r.k, r.type, r.q_stride, r.k_stride, (const float*)r.q_weight,
                                    (const float*)r.k_weight, r.eps, (const float*)r.cos_sin, x.positions, x.stride,
                                    x.count, x.of, r.num_positions, pairing, (float*)r.q_out, k_out,
                                    bf16 ? ATTN_BF16 : ATTN_F32, r.n, st);
    });
  });
}

// bf16 pages, k, v, kPages, vPages, blockTable, contextLens, rowStart, cosSin, positions, axes, kWeight, q, qOut,
// qWeight, eps, pairing, stream
PyObject* append_paged_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("append_paged_axes", n, 18, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Rows r;
    rows(&c, &r, a[12], a[1], Py_None, a[8], a[13], a[14], a[11], a[15]);
    long long vs[3] = {r.n, ATTN_HKV, ATTN_D}, v_stride = 0;
    void* v = tensor(&c, "v", a[2], r.dtype, 3, vs, &v_stride);
    Axes p;
    axes_of(&c, &p, r.n, a[9], a[10]);
    Batch x;
    batch(&c, &x, bf16, a[3], a[4], a[5], a[6]);
    long long st1[1] = {(long long)x.B + 1};
    const int* starts = (const int*)tensor(&c, "rowStart", a[7], kI32, 1, st1);
    const int pairing = integer(&c, "pairing", a[16]);
    const cudaStream_t st = stream_of(&c, a[17]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(r.q, r.k, v, r.type, r.q_stride, r.k_stride, v_stride, (const float*)r.q_weight,
                  (const float*)r.k_weight, r.eps, (const float*)r.cos_sin, p.positions, p.stride, p.count, p.of,
                  r.num_positions, pairing, (float*)r.q_out, k_pages, v_pages, (const int*)x.table, (const int*)x.ctx,
                  starts, x.B, r.n, x.max_blocks, x.num_pages, st);
      };
      return bf16 ? go(attn_append_paged_axes_bf16kv, (uint16_t*)x.k_pages, (uint16_t*)x.v_pages)
                  : go(attn_append_paged_axes, (float*)x.k_pages, (float*)x.v_pages);
    });
  });
}

// bf16 pages, q, kPages, vPages, weights, blockTable, contextLens, out, max_context, decay, weighedLens, workspace, stream
PyObject* decode_weigh_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("decode_weigh_paged", n, 13, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Batch x;
    batch(&c, &x, bf16, a[2], a[3], a[5], a[6], a[4]);
    long long qs[3] = {x.B, ATTN_HQ, ATTN_D}, len[1] = {x.B};
    const float* q = (const float*)tensor(&c, "q", a[1], kF32, 3, qs);
    float* out = (float*)tensor(&c, "out", a[7], kF32, 3, qs);
    const int max_context = integer(&c, "max_context", a[8]);
    const float decay = real(&c, a[9]);
    const int* weighed = (const int*)optional(&c, "weighedLens", a[10], kI32, 1, len);
    size_t bytes = 0;
    void* ws = workspace_of(&c, a[11], &bytes);
    const cudaStream_t st = stream_of(&c, a[12]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(q, k_pages, v_pages, x.weights, (const int*)x.table, (const int*)x.ctx, weighed, decay, out, x.B,
                  x.max_blocks, x.num_pages, max_context, ws, bytes, st);
      };
      return bf16 ? go(attn_decode_weigh_paged_bf16kv, (const uint16_t*)x.k_pages, (const uint16_t*)x.v_pages)
                  : go(attn_decode_weigh_paged, (const float*)x.k_pages, (const float*)x.v_pages);
    });
  });
}

// bf16 pages, q, kPages, weights, blockTable, contextLens, rowStart, max_rows, max_context, decay, weighedLens, workspace,
// stream
PyObject* weigh_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("weigh_paged", n, 13, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Batch x;
    batch(&c, &x, bf16, a[2], nullptr, a[4], a[5], a[3]);
    long long qs[3] = {kAny, ATTN_HQ, ATTN_D}, len[1] = {x.B}, st1[1] = {(long long)x.B + 1};
    const float* q = (const float*)tensor(&c, "q", a[1], kF32, 3, qs);
    const int rows_n = extent(&c, "q", qs[0]);
    const int* starts = (const int*)tensor(&c, "rowStart", a[6], kI32, 1, st1);
    const int max_rows = integer(&c, "max_rows", a[7]), max_context = integer(&c, "max_context", a[8]);
    const float decay = real(&c, a[9]);
    const int* weighed = (const int*)optional(&c, "weighedLens", a[10], kI32, 1, len);
    size_t bytes = 0;
    void* ws = workspace_of(&c, a[11], &bytes);
    const cudaStream_t st = stream_of(&c, a[12]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages) {
        return fn(q, k_pages, x.weights, (const int*)x.table, (const int*)x.ctx, starts, weighed, decay, x.B, rows_n,
                  max_rows, x.max_blocks, x.num_pages, max_context, ws, bytes, st);
      };
      return bf16 ? go(attn_weigh_paged_bf16kv, (const uint16_t*)x.k_pages) : go(attn_weigh_paged, (const float*)x.k_pages);
    });
  });
}

// bf16 pages, kPages, vPages, weights, blockTable, contextLens, keepLens, max_context, keep_first, keep_last, workspace,
// stream
PyObject* evict_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("evict_paged", n, 12, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Batch x;
    batch(&c, &x, bf16, a[1], a[2], a[4], a[5], a[3]);
    long long len[1] = {x.B};
    const int* keep = (const int*)tensor(&c, "keepLens", a[6], kI32, 1, len);
    const int max_context = integer(&c, "max_context", a[7]), first = integer(&c, "keep_first", a[8]),
              last = integer(&c, "keep_last", a[9]);
    size_t bytes = 0;
    void* ws = workspace_of(&c, a[10], &bytes);
    const cudaStream_t st = stream_of(&c, a[11]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(k_pages, v_pages, x.weights, (const int*)x.table, (const int*)x.ctx, keep, first, last, x.B,
                  x.max_blocks, x.num_pages, max_context, ws, bytes, st);
      };
      return bf16 ? go(attn_evict_paged_bf16kv, (uint16_t*)x.k_pages, (uint16_t*)x.v_pages)
                  : go(attn_evict_paged, (float*)x.k_pages, (float*)x.v_pages);
    });
  });
}

// bf16 pages, q, kPages, vPages, blockTable, contextLens, rowStart, masks, out, max_rows, max_context, num_splits,
// workspace, stream
PyObject* tree_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("tree_paged", n, 14, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    long long qs[3] = {kAny, ATTN_HQ, ATTN_D};
    const float* q = (const float*)tensor(&c, "q", a[1], kF32, 3, qs);
    float* out = (float*)tensor(&c, "out", a[8], kF32, 3, qs);
    const int rows_n = extent(&c, "q", qs[0]);
    Batch x;
    batch(&c, &x, bf16, a[2], a[3], a[4], a[5]);
    long long st1[1] = {(long long)x.B + 1}, ms[1] = {qs[0]};
    const int* starts = (const int*)tensor(&c, "rowStart", a[6], kI32, 1, st1);
    const long long* masks = (const long long*)optional(&c, "masks", a[7], kI64, 1, ms);
    const int max_rows = integer(&c, "max_rows", a[9]), max_context = integer(&c, "max_context", a[10]),
              splits = integer(&c, "num_splits", a[11]);
    size_t bytes = 0;
    void* ws = workspace_of(&c, a[12], &bytes);
    const cudaStream_t st = stream_of(&c, a[13]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(q, k_pages, v_pages, (const int*)x.table, (const int*)x.ctx, starts, masks, out, x.B, rows_n, max_rows,
                  x.max_blocks, x.num_pages, max_context, splits, ws, bytes, st);
      };
      return bf16 ? go(attn_tree_paged_bf16kv, (const uint16_t*)x.k_pages, (const uint16_t*)x.v_pages)
                  : go(attn_tree_paged, (const float*)x.k_pages, (const float*)x.v_pages);
    });
  });
}

// bf16 pages, kPages, vPages, blockTable, contextLens, keep, keepCounts, max_rows, stream
PyObject* compact_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return entry("compact_paged", n, 9, [&]() -> PyObject* {
    Call c;
    const bool bf16 = a[0] == Py_True;
    Batch x;
    batch(&c, &x, bf16, a[1], a[2], a[3], a[4]);
    long long ks[2] = {x.B, kAny}, cs[1] = {x.B};
    const int* keep = (const int*)tensor(&c, "keep", a[5], kI32, 2, ks);
    const int* counts = (const int*)tensor(&c, "keepCounts", a[6], kI32, 1, cs);
    const int max_keep = extent(&c, "keep", ks[1]), max_rows = integer(&c, "max_rows", a[7]);
    const cudaStream_t st = stream_of(&c, a[8]);
    return call(c, [&] {
      const auto go = [&](auto fn, auto* k_pages, auto* v_pages) {
        return fn(k_pages, v_pages, (const int*)x.table, (const int*)x.ctx, keep, counts, x.B, max_keep, max_rows,
                  x.max_blocks, x.num_pages, st);
      };
      return bf16 ? go(attn_compact_paged_bf16kv, (uint16_t*)x.k_pages, (uint16_t*)x.v_pages)
                  : go(attn_compact_paged, (float*)x.k_pages, (float*)x.v_pages);
    });
  });
}

PyMethodDef methods[] = {
    {"qk_norm_rope", (PyCFunction)(void (*)(void))qk_norm_rope, METH_FASTCALL, "attn_qk_norm_rope"},
    {"append_paged", (PyCFunction)(void (*)(void))append_paged, METH_FASTCALL, "attn_append_paged(_bf16kv)"},
    {"qk_norm_rope_axes", (PyCFunction)(void (*)(void))qk_norm_rope_axes, METH_FASTCALL, "attn_qk_norm_rope_axes"},
    {"append_paged_axes", (PyCFunction)(void (*)(void))append_paged_axes, METH_FASTCALL, "attn_append_paged_axes(_bf16kv)"},
    {"decode_weigh_paged", (PyCFunction)(void (*)(void))decode_weigh_paged, METH_FASTCALL, "attn_decode_weigh_paged(_bf16kv)"},
    {"weigh_paged", (PyCFunction)(void (*)(void))weigh_paged, METH_FASTCALL, "attn_weigh_paged(_bf16kv)"},
    {"evict_paged", (PyCFunction)(void (*)(void))evict_paged, METH_FASTCALL, "attn_evict_paged(_bf16kv)"},
    {"tree_paged", (PyCFunction)(void (*)(void))tree_paged, METH_FASTCALL, "attn_tree_paged(_bf16kv)"},
    {"compact_paged", (PyCFunction)(void (*)(void))compact_paged, METH_FASTCALL, "attn_compact_paged(_bf16kv)"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "argument marshalling of the serving-step calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
