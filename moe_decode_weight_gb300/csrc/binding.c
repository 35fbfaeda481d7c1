/* Marshalling of the calls of the attention sub-layers and the norm between them, as a CPython extension (module _binding).
 *
 * A window's calls take a few microseconds on the GPU, and reading ten tensors' types, shapes, strides and
 * addresses from Python takes longer than that: a call of mdw_kv_plan took 10.1 us, of which the library's
 * part was 3.2 us, and takes 6.0 us through this module (mdw_tree_attention 13.3 -> 7.6, w4_linear 7.5 -> 4.1,
 * mdw_kv_write 7.1 -> 4.1). It does the checks that the Python code did and calls the library's entry points, whose addresses
 * the package hands it; it holds no arithmetic and keeps nothing of its arguments. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "moe_decode_weight.h"

enum { T_BF16 = 1, T_F16 = 2, T_F32 = 4, T_E4M3 = 8, T_U8 = 16, T_I32 = 32, T_I64 = 64, T_U64 = 128, T_KINDS = 8 };

static PyObject *g_types[T_KINDS], *g_refuse, *g_device, *g_stream;
static PyObject *s_dtype, *s_data_ptr, *s_get_device, *s_shape, *s_stride, *s_address, *s_device_index, *s_cuda_stream, *s_is_contiguous;

typedef mdw_status (*w4_fn)(const mdw_w4_weights*, int32_t, const void*, int64_t, void*, int64_t, int32_t, const void*, const void*,
                            int64_t, uint32_t*, mdw_stream_t);
typedef mdw_status (*plan_fn)(int32_t, const int32_t*, const int32_t*, int32_t, int32_t, int32_t*, int32_t, const int32_t*, int32_t,
                              const int32_t*, int32_t, int32_t*, int64_t*, int32_t*, uint64_t*, int32_t*, uint32_t*, mdw_stream_t);
typedef mdw_status (*write_fn)(const mdw_kv_cache*, int32_t, const void*, int64_t, const void*, int64_t, int32_t, const int64_t*,
                               uint32_t*, mdw_stream_t);
typedef mdw_status (*attention_fn)(const mdw_kv_cache*, int32_t, int32_t, int32_t, int32_t, const void*, int64_t, int32_t, void*,
                                   int64_t, float*, const int32_t*, int32_t, const int32_t*, const int32_t*, const uint64_t*, float,
                                   uint32_t*, void*, size_t, mdw_stream_t);
typedef mdw_status (*linear_fn)(const mdw_linear_state*, int32_t, int32_t, int32_t, int32_t, const void*, int64_t, const void*, int64_t,
                                const void*, int64_t, const float*, int64_t, void*, int64_t, const int32_t*, const int32_t*,
                                const int32_t*, float, uint32_t*, void*, size_t, mdw_stream_t);
typedef mdw_status (*linear_tree_fn)(const mdw_linear_state*, int32_t, int32_t, int32_t, int32_t, const void*, int64_t, const void*,
                                     int64_t, const void*, int64_t, const float*, int64_t, void*, int64_t, const int32_t*,
                                     const int32_t*, const uint64_t*, float, uint32_t*, mdw_stream_t);
typedef mdw_status (*advance_fn)(const mdw_linear_state*, int32_t, int32_t, int32_t, int32_t, const void*, int64_t, const void*, int64_t,
                                 const float*, int64_t, const int32_t*, const uint64_t*, const int32_t*, const int32_t*, uint32_t*,
                                 mdw_stream_t);
typedef mdw_status (*norm_fn)(int32_t, int32_t, int32_t, const void*, int64_t, int32_t, const void*, int32_t, const void*, int64_t,
                              int32_t, float, const void*, int64_t, float, void*, int64_t, int32_t, const void*, void*, int64_t, float,
                              mdw_stream_t);
static w4_fn g_w4;
static plan_fn g_plan;
static write_fn g_write;
static attention_fn g_attention;
static linear_fn g_linear;
static linear_tree_fn g_linear_tree;
static advance_fn g_advance;
static norm_fn g_norm;

/* One call's state: the device of its handle or first tensor, which the others have to share. */
typedef struct {
  const char* fn;
  long device;
} Call;

typedef struct {
  void* p;
  int type, dims;
  int64_t size[4], stride[4];
} Tensor;

/* Raises the package's error with a status code. */
static int refuse(const Call* c, int code, const char* name, const char* detail) {
  PyObject* e = PyObject_CallFunction(g_refuse, "siN", c->fn, code, PyUnicode_FromFormat("%s %s", name, detail));
  if (e) {
    PyErr_SetObject((PyObject*)Py_TYPE(e), e);
    Py_DECREF(e);
  }
  return 0;
}

static int number(PyObject* o, int64_t* out) {
  *out = o ? PyLong_AsLongLong(o) : -1;
  Py_XDECREF(o);
  return !PyErr_Occurred();
}
static int numbers(PyObject* tuple, int64_t* out, int* n) {
  if (!tuple) return 0;
  const Py_ssize_t k = PyTuple_Check(tuple) ? PyTuple_GET_SIZE(tuple) : 5;
  if (k > 4) {
    *n = 5;
  } else {
    *n = (int)k;
    for (Py_ssize_t i = 0; i < k; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  }
  Py_DECREF(tuple);
  return !PyErr_Occurred();
}

/* Reads a tensor of one of the `types`, with or without its strides; None (if `optional`) gives a null pointer. */
static int tensor(Call* c, PyObject* t, const char* name, int types, int optional, int strides, Tensor* out) {
  memset(out, 0, sizeof *out);
  if (t == Py_None && optional) return 1;
  PyObject* type = PyObject_GetAttr(t, s_dtype);
  if (!type) return 0;
  for (int i = 0; i < T_KINDS; ++i)
    if (type == g_types[i]) out->type = 1 << i;
  Py_DECREF(type);
  int64_t device, p;
  int n;
  if (!number(PyObject_CallMethodNoArgs(t, s_get_device), &device) || !number(PyObject_CallMethodNoArgs(t, s_data_ptr), &p) ||
      !numbers(PyObject_GetAttr(t, s_shape), out->size, &out->dims) ||
      (strides && !numbers(PyObject_CallMethodNoArgs(t, s_stride), out->stride, &n)))
    return 0;
  if (device < 0) return refuse(c, MDW_ERR_INVALID_ARG, name, "has to be on a CUDA device");
  if (!(out->type & types)) return refuse(c, MDW_ERR_FORMAT_MISMATCH, name, "has another type than the call takes");
  if (c->device < 0) c->device = (long)device;
  if (device != c->device) return refuse(c, MDW_ERR_INVALID_ARG, name, "is on another device");
  if (out->dims > 4) return refuse(c, MDW_ERR_INVALID_ARG, name, "has too many dimensions");
  out->p = (void*)(intptr_t)p;
  return 1;
}
/* Whether the elements of a row are laid out without gaps. */
static int packed_rows(const Tensor* t) {
  int64_t width = 1;
  for (int i = t->dims - 1; i > 0; --i) {
    if (t->size[i] != 1 && t->stride[i] != width) return 0;
    width *= t->size[i];
  }
  return 1;
}
/* A contiguous array; want: its sizes (-1: any), of which there are `dims`. */
static int array(Call* c, PyObject* o, const char* name, int types, int optional, int dims, int64_t d0, int64_t d1, Tensor* out) {
  if (!tensor(c, o, name, types, optional, 0, out)) return 0;
  if (o == Py_None) return 1;
  PyObject* r = PyObject_CallMethodNoArgs(o, s_is_contiguous);
  if (!r) return 0;
  const int contiguous = r == Py_True;
  Py_DECREF(r);
  if (out->dims != dims || (d0 >= 0 && out->size[0] != d0) || (dims > 1 && d1 >= 0 && out->size[1] != d1) || !contiguous)
    return refuse(c, MDW_ERR_INVALID_ARG, name, "has another shape, or is not contiguous");
  return 1;
}
/* Rows [d0][d1](...[d2]) with contiguous elements; *ld their stride. */
static int rows(Call* c, PyObject* o, const char* name, int types, int optional, int dims, int64_t d0, int64_t d1, int64_t d2, Tensor* out,
                int64_t* ld) {
  *ld = 0;
  if (!tensor(c, o, name, types, optional, 1, out)) return 0;
  if (o == Py_None) return 1;
  if (out->dims != dims || (d0 >= 0 && out->size[0] != d0) || (d1 >= 0 && out->size[1] != d1) || (dims > 2 && d2 >= 0 && out->size[2] != d2) ||
      !packed_rows(out))
    return refuse(c, MDW_ERR_INVALID_ARG, name, "has another shape, or rows whose elements are not contiguous");
  const int64_t width = out->size[1] * (dims > 2 ? out->size[2] : 1);
  *ld = out->size[0] != 1 ? out->stride[0] : (width + 7) / 8 * 8;
  return 1;
}
/* Address of a weight or cache handle's descriptor, whose first two words are the magic and the format; the call's
 * tensors have to be on its device. */
static const void* handle(Call* c, PyObject* o, uint32_t format) {
  int64_t a, device;
  if (!number(PyObject_GetAttr(o, s_address), &a) || !number(PyObject_GetAttr(o, s_device_index), &device)) return NULL;
  c->device = (long)device;
  const uint32_t* d = (const uint32_t*)(intptr_t)a;
  if (d[0] == MDW_MAGIC && d[1] == format) return d;
  refuse(c, MDW_ERR_FORMAT_MISMATCH, "the handle", "is of another kind");
  return NULL;
}
/* The stream to launch on, given or the device's current one. Returns 0 with no error set if the tensors' device is not
 * the current one (the package then makes it so and calls again). */
static int stream_of(const Call* c, PyObject* given, mdw_stream_t* out, int* elsewhere) {
  int64_t device, s;
  *elsewhere = 0;
  if (!number(PyObject_CallNoArgs(g_device), &device)) return 0;
  if (device != c->device) {
    *elsewhere = 1;
    return 0;
  }
  if (given != Py_None) {
    if (!number(PyObject_GetAttr(given, s_cuda_stream), &s)) return 0;
  } else {
    PyObject* d = PyLong_FromLong(c->device);
    PyObject* r = d ? PyObject_CallOneArg(g_stream, d) : NULL;
    Py_XDECREF(d);
    if (!number(r, &s)) return 0;
  }
  *out = (mdw_stream_t)(intptr_t)s;
  return 1;
}
static int fits32(int64_t v) { return v >= 0 && v <= INT32_MAX; }
/* None after a call that was made, the device's index if it has to become the current one first. */
static PyObject* result(const Call* c, int elsewhere, mdw_status st) {
  if (elsewhere) return PyLong_FromLong(c->device);
  if (st != MDW_OK) {
    PyObject* e = PyObject_CallFunction(g_refuse, "sis", c->fn, (int)st, "");
    if (e) {
      PyErr_SetObject((PyObject*)Py_TYPE(e), e);
      Py_DECREF(e);
    }
    return NULL;
  }
  Py_RETURN_NONE;
}
static int dtype_code(int t) { return t == T_BF16 ? MDW_DT_BF16 : t == T_F16 ? MDW_DT_F16 : t == T_F32 ? MDW_DT_F32 : MDW_DT_E4M3; }
static int arguments(const char* fn, Py_ssize_t got, Py_ssize_t wanted) {
  if (got == wanted) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, wanted, got);
  return 0;
}

/* w4_linear(handle, x, y, bias, residual, status, stream) */
static PyObject* b_w4_linear(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"w4_linear", -1};
  Tensor x, y, bias, res, status;
  int64_t ldx, ldy, ldr;
  const mdw_w4_weights* w;
  if (!arguments(c.fn, n, 7) || !(w = handle(&c, a[0], MDW_FMT_INT4_GROUP))) return NULL;
  const int type = w->dtype == MDW_DT_BF16 ? T_BF16 : T_F16;
  if (!rows(&c, a[1], "x", type, 0, 2, -1, w->k, 0, &x, &ldx) || !rows(&c, a[2], "y", type | T_F32, 0, 2, x.size[0], w->n, 0, &y, &ldy) ||
      !array(&c, a[3], "bias", type, 1, 1, w->n, 0, &bias) || !rows(&c, a[4], "residual", type, 1, 2, x.size[0], w->n, 0, &res, &ldr) ||
      !array(&c, a[5], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[6], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  const int m = fits32(x.size[0]) ? (int)x.size[0] : 0;
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_w4(w, m, x.p, ldx, y.p, ldy, dtype_code(y.type), bias.p, res.p, ldr, status.p, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* kv_plan(ctx_len, new_len, page_size, num_pages, block_table, free_pages, row_start, slot_map, positions, pages_taken, parents,
 * tree_mask, status, stream) */
static PyObject* b_kv_plan(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_kv_plan", -1};
  Tensor ctx, add, table, fr, start, slot, pos, taken, parents, mask, status;
  if (!arguments(c.fn, n, 14)) return NULL;
  if (!array(&c, a[0], "ctx_len", T_I32, 0, 1, -1, 0, &ctx)) return NULL;
  const int64_t b = ctx.size[0];
  if (!array(&c, a[1], "new_len", T_I32, 0, 1, b, 0, &add) || !array(&c, a[4], "block_table", T_I32, 0, 2, b, -1, &table) ||
      !array(&c, a[5], "free_pages", T_I32, 0, 1, -1, 0, &fr) || !array(&c, a[6], "row_start", T_I32, 0, 1, b + 1, 0, &start) ||
      !array(&c, a[7], "slot_map", T_I64, 0, 1, -1, 0, &slot))
    return NULL;
  const int64_t t = slot.size[0];
  if (!array(&c, a[8], "positions", T_I32, 0, 1, t, 0, &pos) || !array(&c, a[9], "pages_taken", T_I32, 0, 1, 1, 0, &taken) ||
      !array(&c, a[10], "parents", T_I32, 1, 1, t, 0, &parents) || !array(&c, a[11], "tree_mask", T_I64 | T_U64, 1, 1, t, 0, &mask) ||
      !array(&c, a[12], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  const int64_t page = PyLong_AsLongLong(a[2]), pages = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[13], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(b) || !fits32(page) || !fits32(pages) || !fits32(table.size[1]) || !fits32(fr.size[0]) || !fits32(t))
    return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_plan((int)b, ctx.p, add.p, (int)page, (int)pages, table.p, (int)table.size[1], fr.p, (int)fr.size[0], parents.p, (int)t,
                              start.p, slot.p, pos.p, mask.p, taken.p, status.p, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* kv_write(handle, k, v, slot_map, status, stream) */
static PyObject* b_kv_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_kv_write", -1};
  Tensor k, v, slot, status;
  int64_t ldk, ldv;
  const mdw_kv_cache* h;
  if (!arguments(c.fn, n, 6) || !(h = handle(&c, a[0], MDW_FMT_KV_PAGED))) return NULL;
  if (!rows(&c, a[1], "k", T_BF16 | T_F16, 0, 3, -1, h->kv_heads, h->head_dim, &k, &ldk) ||
      !rows(&c, a[2], "v", k.type, 0, 3, k.size[0], h->kv_heads, h->head_dim, &v, &ldv) ||
      !array(&c, a[3], "slot_map", T_I64, 0, 1, k.size[0], 0, &slot) || !array(&c, a[4], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[5], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  const int t = fits32(k.size[0]) ? (int)k.size[0] : 0;
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_write(h, t, k.p, ldk, v.p, ldv, dtype_code(k.type), slot.p, status.p, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* tree_attention(handle, q, out, block_table, ctx_len, row_start, max_new, ws, tree_mask, lse, scale, status, stream) */
static PyObject* b_tree_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_tree_attention", -1};
  Tensor q, out, table, ctx, start, ws, mask, lse, status;
  int64_t ldq, ldo;
  const mdw_kv_cache* h;
  if (!arguments(c.fn, n, 13) || !(h = handle(&c, a[0], MDW_FMT_KV_PAGED))) return NULL;
  if (!rows(&c, a[1], "q", T_BF16 | T_F16, 0, 3, -1, -1, h->head_dim, &q, &ldq) ||
      !rows(&c, a[2], "out", q.type, 0, 3, q.size[0], q.size[1], h->head_dim, &out, &ldo) ||
      !array(&c, a[4], "ctx_len", T_I32, 0, 1, -1, 0, &ctx))
    return NULL;
  const int64_t b = ctx.size[0];
  if (!array(&c, a[3], "block_table", T_I32, 0, 2, b, -1, &table) || !array(&c, a[5], "row_start", T_I32, 0, 1, b + 1, 0, &start) ||
      !array(&c, a[7], "ws", T_U8, 0, 1, -1, 0, &ws) || !array(&c, a[8], "tree_mask", T_I64 | T_U64, 1, 1, q.size[0], 0, &mask) ||
      !array(&c, a[9], "lse", T_F32, 1, 2, q.size[0], q.size[1], &lse) || !array(&c, a[11], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  const int64_t most = PyLong_AsLongLong(a[6]);
  const double scale = a[10] == Py_None ? 1.0 / sqrt((double)h->head_dim) : PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[12], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(b) || !fits32(q.size[0]) || !fits32(q.size[1]) || !fits32(most) || !fits32(table.size[1])) return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_attention(h, (int)b, (int)q.size[0], (int)q.size[1], (int)most, q.p, ldq, dtype_code(q.type), out.p, ldo, lse.p, table.p,
                                   (int)table.size[1], ctx.p, start.p, mask.p, (float)scale, status.p, ws.p, (size_t)ws.size[0], s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* Log decays [T][heads] with contiguous elements, or [heads] for all rows (*ld = 0). */
static int decays(Call* c, PyObject* o, int64_t t, int64_t heads, Tensor* out, int64_t* ld) {
  *ld = 0;
  if (!tensor(c, o, "log_decay", T_F32, 0, 1, out)) return 0;
  const int one = out->dims == 1;
  if ((out->dims != 1 && out->dims != 2) || out->size[out->dims - 1] != heads || (heads > 1 && out->stride[out->dims - 1] != 1) ||
      (!one && out->size[0] != t))
    return refuse(c, MDW_ERR_INVALID_ARG, "log_decay", "has another shape, or heads that are not contiguous");
  if (!one) *ld = t == 1 ? heads : out->stride[0];
  return 1;
}

/* linear_attention(handle, q, k, v, log_decay, out, row_start, slot_in, slot_out, max_new, ws, scale, status, stream) */
static PyObject* b_linear_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_linear_attention", -1};
  Tensor q, k, v, g, out, start, in, to, ws, status;
  int64_t ldq, ldk, ldv, ldd, ldo;
  const mdw_linear_state* h;
  if (!arguments(c.fn, n, 14) || !(h = handle(&c, a[0], MDW_FMT_LINEAR_STATE))) return NULL;
  if (!rows(&c, a[1], "q", T_BF16, 0, 3, -1, -1, h->head_dim, &q, &ldq)) return NULL;
  const int64_t t = q.size[0];
  if (!rows(&c, a[2], "k", T_BF16, 0, 3, t, q.size[1], h->head_dim, &k, &ldk) ||
      !rows(&c, a[3], "v", T_BF16, 0, 3, t, h->heads, h->head_dim, &v, &ldv) || !decays(&c, a[4], t, h->heads, &g, &ldd) ||
      !rows(&c, a[5], "out", T_BF16, 0, 3, t, h->heads, h->head_dim, &out, &ldo) ||
      !array(&c, a[7], "slot_in", T_I32, 0, 1, -1, 0, &in) || !array(&c, a[6], "row_start", T_I32, 0, 1, in.size[0] + 1, 0, &start) ||
      !array(&c, a[8], "slot_out", T_I32, 0, 1, in.size[0], 0, &to) || !array(&c, a[10], "ws", T_U8, 0, 1, -1, 0, &ws) ||
      !array(&c, a[12], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  const int64_t most = PyLong_AsLongLong(a[9]);
  const double scale = a[11] == Py_None ? 1.0 / sqrt((double)h->head_dim) : PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[13], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(in.size[0]) || !fits32(t) || !fits32(q.size[1]) || !fits32(most)) return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_linear(h, (int)in.size[0], (int)t, (int)q.size[1], (int)most, q.p, ldq, k.p, ldk, v.p, ldv, g.p, ldd, out.p, ldo, start.p, in.p,
                to.p, (float)scale, status.p, ws.p, (size_t)ws.size[0], s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* linear_tree_attention(handle, q, k, v, log_decay, out, row_start, slot_in, max_new, tree_mask, scale, status, stream) */
static PyObject* b_linear_tree(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_linear_tree_attention", -1};
  Tensor q, k, v, g, out, start, in, mask, status;
  int64_t ldq, ldk, ldv, ldd, ldo;
  const mdw_linear_state* h;
  if (!arguments(c.fn, n, 13) || !(h = handle(&c, a[0], MDW_FMT_LINEAR_STATE))) return NULL;
  if (!rows(&c, a[1], "q", T_BF16, 0, 3, -1, -1, h->head_dim, &q, &ldq)) return NULL;
  const int64_t t = q.size[0];
  if (!rows(&c, a[2], "k", T_BF16, 0, 3, t, q.size[1], h->head_dim, &k, &ldk) ||
      !rows(&c, a[3], "v", T_BF16, 0, 3, t, h->heads, h->head_dim, &v, &ldv) || !decays(&c, a[4], t, h->heads, &g, &ldd) ||
      !rows(&c, a[5], "out", T_BF16, 0, 3, t, h->heads, h->head_dim, &out, &ldo) ||
      !array(&c, a[7], "slot_in", T_I32, 0, 1, -1, 0, &in) || !array(&c, a[6], "row_start", T_I32, 0, 1, in.size[0] + 1, 0, &start) ||
      !array(&c, a[9], "tree_mask", T_I64 | T_U64, 1, 1, t, 0, &mask) || !array(&c, a[11], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  const int64_t most = PyLong_AsLongLong(a[8]);
  const double scale = a[10] == Py_None ? 1.0 / sqrt((double)h->head_dim) : PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[12], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(in.size[0]) || !fits32(t) || !fits32(q.size[1]) || !fits32(most)) return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_linear_tree(h, (int)in.size[0], (int)t, (int)q.size[1], (int)most, q.p, ldq, k.p, ldk, v.p, ldv, g.p, ldd, out.p, ldo, start.p,
                     in.p, mask.p, (float)scale, status.p, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* linear_state_advance(handle, k, v, log_decay, row_start, accepted, slot_in, slot_out, max_new, status, stream) */
static PyObject* b_linear_advance(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_linear_state_advance", -1};
  Tensor k, v, g, start, take, in, to, status;
  int64_t ldk, ldv, ldd;
  const mdw_linear_state* h;
  if (!arguments(c.fn, n, 11) || !(h = handle(&c, a[0], MDW_FMT_LINEAR_STATE))) return NULL;
  if (!rows(&c, a[1], "k", T_BF16, 0, 3, -1, -1, h->head_dim, &k, &ldk)) return NULL;
  const int64_t t = k.size[0];
  if (!rows(&c, a[2], "v", T_BF16, 0, 3, t, h->heads, h->head_dim, &v, &ldv) || !decays(&c, a[3], t, h->heads, &g, &ldd) ||
      !array(&c, a[6], "slot_in", T_I32, 0, 1, -1, 0, &in) || !array(&c, a[4], "row_start", T_I32, 0, 1, in.size[0] + 1, 0, &start) ||
      !array(&c, a[5], "accepted", T_I64 | T_U64, 0, 1, in.size[0], 0, &take) || !array(&c, a[7], "slot_out", T_I32, 0, 1, in.size[0], 0, &to) ||
      !array(&c, a[9], "status", T_I32, 1, 1, 1, 0, &status))
    return NULL;
  const int64_t most = PyLong_AsLongLong(a[8]);
  if (PyErr_Occurred()) return NULL;
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[10], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(in.size[0]) || !fits32(t) || !fits32(k.size[1]) || !fits32(most)) return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_advance(h, (int)in.size[0], (int)t, (int)k.size[1], (int)most, k.p, ldk, v.p, ldv, g.p, ldd, start.p, take.p, in.p, to.p, status.p, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* block_norm(y, sum, post_weight, group, gate, gate kind, residual, pre_weight, x, branch_scale, residual_scale, eps, stream) */
static PyObject* b_block_norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  Call c = {"mdw_block_norm", -1};
  Tensor y, sum, post, gate, res, pre, x;
  int64_t ldy, lds, ldr, ldx, ldg = 0;
  if (!arguments(c.fn, n, 13) || !rows(&c, a[0], "y", T_BF16 | T_F16 | T_F32, 0, 2, -1, -1, 0, &y, &ldy)) return NULL;
  const int64_t t = y.size[0], w = y.size[1];
  const int64_t group = a[3] == Py_None ? w : PyLong_AsLongLong(a[3]), kind = PyLong_AsLongLong(a[5]);
  const double fb = PyFloat_AsDouble(a[9]), fr = PyFloat_AsDouble(a[10]), eps = PyFloat_AsDouble(a[11]);
  if (PyErr_Occurred()) return NULL;
  const int any = T_BF16 | T_F16;
  if (!tensor(&c, a[4], "gate", any, 1, 1, &gate) || !array(&c, a[2], "post_weight", any, 1, 1, group, 0, &post) ||
      !rows(&c, a[8], "x", any, 1, 2, t, w, 0, &x, &ldx) || !array(&c, a[7], "pre_weight", any, 1, 1, w, 0, &pre) ||
      !rows(&c, a[1], "sum", any | T_F32, 1, 2, t, w, 0, &sum, &lds) || !rows(&c, a[6], "residual", any | T_F32, 1, 2, t, w, 0, &res, &ldr))
    return NULL;
  if (gate.p || gate.dims) {
    const int last = gate.dims - 1;
    if (gate.dims < 1 || gate.dims > 2 || gate.size[last] != w || (w > 1 && gate.stride[last] != 1) || (gate.dims == 2 && gate.size[0] != t)) {
      refuse(&c, MDW_ERR_INVALID_ARG, "gate", "has another shape, or rows whose elements are not contiguous");
      return NULL;
    }
    if (gate.dims == 2) ldg = t == 1 ? (w + 7) / 8 * 8 : gate.stride[0];
  }
  /* the 16-bit type: that of the first tensor that has one; the others have to be of it */
  const int types[6] = {y.type, post.type, gate.type, pre.type, x.type, sum.type};
  int type = 0;
  for (int i = 0; i < 6 && !type; ++i) type = types[i] & any;
  if (!type) type = res.type & any ? res.type : T_BF16;
  const int all16 = post.type | gate.type | pre.type | x.type | ((y.type | sum.type | res.type) & any);
  if (all16 & ~type) {
    refuse(&c, MDW_ERR_FORMAT_MISMATCH, "the tensors", "are of two 16-bit types");
    return NULL;
  }
  /* (a sum that nothing stores is not rounded before x) */
  const int sums = sum.type ? sum.type : res.type ? res.type : x.type ? T_F32 : type;
  if (res.type && res.type != sums) {
    refuse(&c, MDW_ERR_FORMAT_MISMATCH, "residual", "has another type than sum");
    return NULL;
  }
  mdw_stream_t s;
  int elsewhere;
  if (!stream_of(&c, a[12], &s, &elsewhere)) return elsewhere ? result(&c, 1, MDW_OK) : NULL;
  if (!fits32(t) || !fits32(w) || !fits32(group)) return result(&c, 0, MDW_ERR_INVALID_ARG);
  mdw_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_norm((int)t, (int)w, dtype_code(type), y.p, ldy, dtype_code(y.type), post.p, (int)group, gate.p, ldg, (int)kind, (float)fb, res.p, ldr,
              (float)fr, sum.p, lds, dtype_code(sums), pre.p, x.p, ldx, (float)eps, s);
  Py_END_ALLOW_THREADS;
  return result(&c, 0, st);
}

/* setup(types, refuse, current device, current stream, addresses of the eight entry points) */
static PyObject* b_setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (!arguments("setup", n, 5)) return NULL;
  if (!PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != T_KINDS || !PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 8) {
    PyErr_SetString(PyExc_TypeError, "setup: types and addresses are tuples of 8 each");
    return NULL;
  }
  void* f[8];
  for (int i = 0; i < 8; ++i) f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[4], i));
  if (PyErr_Occurred()) return NULL;
  for (int i = 0; i < T_KINDS; ++i) Py_XSETREF(g_types[i], Py_NewRef(PyTuple_GET_ITEM(a[0], i)));
  Py_XSETREF(g_refuse, Py_NewRef(a[1]));
  Py_XSETREF(g_device, Py_NewRef(a[2]));
  Py_XSETREF(g_stream, Py_NewRef(a[3]));
  g_w4 = (w4_fn)f[0];
  g_plan = (plan_fn)f[1];
  g_write = (write_fn)f[2];
  g_attention = (attention_fn)f[3];
  g_linear = (linear_fn)f[4];
  g_linear_tree = (linear_tree_fn)f[5];
  g_advance = (advance_fn)f[6];
  g_norm = (norm_fn)f[7];
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))b_setup, METH_FASTCALL, NULL},
                                {"w4_linear", (PyCFunction)(void (*)(void))b_w4_linear, METH_FASTCALL, NULL},
                                {"kv_plan", (PyCFunction)(void (*)(void))b_kv_plan, METH_FASTCALL, NULL},
                                {"kv_write", (PyCFunction)(void (*)(void))b_kv_write, METH_FASTCALL, NULL},
                                {"tree_attention", (PyCFunction)(void (*)(void))b_tree_attention, METH_FASTCALL, NULL},
                                {"linear_attention", (PyCFunction)(void (*)(void))b_linear_attention, METH_FASTCALL, NULL},
                                {"linear_tree_attention", (PyCFunction)(void (*)(void))b_linear_tree, METH_FASTCALL, NULL},
                                {"linear_state_advance", (PyCFunction)(void (*)(void))b_linear_advance, METH_FASTCALL, NULL},
                                {"block_norm", (PyCFunction)(void (*)(void))b_block_norm, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_address = PyUnicode_InternFromString("address");
  s_device_index = PyUnicode_InternFromString("device_index");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  return PyModule_Create(&module);
}
