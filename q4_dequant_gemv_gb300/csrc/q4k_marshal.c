/* q4k_marshal.c -- the Python side of q4k_rope, q4k_kv_append, q4k_paged_attention
 * and their forms for an 8-bit cache: checks tensors, fills the structures of include/q4k.h and
 * calls the library.  These calls sit between the launches of a decode step, and
 * reading some forty tensor attributes from Python took 8 to 12 us a call, more
 * than the kernels; here they take a third of that.  Plain CPython API: torch's
 * objects (the Tensor class, dtypes, empty) come in through setup(), the library's
 * functions as addresses. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>
#include <string.h>

#include "q4k.h"

typedef q4k_status (*rope_fn)(const q4k_rope_args *, void *);
typedef q4k_status (*append_fn)(const q4k_paged_cache *, const q4k_append_args *, void *);
typedef q4k_status (*attention_fn)(const q4k_paged_cache *, const q4k_attention_args *, void *);

static PyObject *g_tensor, *g_dtype[3], *g_int32, *g_empty, *g_empty_like, *g_new_on, *g_device, *g_stream_of, *g_raise;
static rope_fn g_rope;
static append_fn g_append;
static attention_fn g_attention;
/* The calls of an 8-bit cache come in by themselves (setup8). */
typedef q4k_status (*norm_rope_fn)(const q4k_norm_rope_args *, void *);
typedef q4k_status (*append8_fn)(const q4k_paged_cache8 *, const q4k_append8_args *, void *);
typedef q4k_status (*attention8_fn)(const q4k_paged_cache8 *, const q4k_attention_args *, void *);
typedef q4k_status (*read8_fn)(const q4k_paged_cache8 *, const q4k_read8_args *, void *);
static PyObject *g_int8, *g_e4m3;
static norm_rope_fn g_norm_rope;
static append8_fn g_append8;
static read8_fn g_read8;
static attention8_fn g_attention8;
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_get_device, *s_device,
    *s_cuda_stream, *k_dtype_device;

/* ---- attributes */

static int is_tensor(PyObject *t, const char *name)
{
    if (PyObject_TypeCheck(t, (PyTypeObject *)g_tensor)) return 1;
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return 0;
}

/* Type code of a tensor's dtype, -1 for another one, -2 with an error set. */
static int dtype_code(PyObject *dtype)
{
    for (int i = 0; i < 3; ++i)
        if (dtype == g_dtype[i]) return i;
    return -1;
}

static PyObject *dtype_of(PyObject *t) /* borrowed: dtypes live as long as torch */
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    Py_XDECREF(d);
    return d;
}

/* Whether t is on the GPU *dev (-1: the first tensor of a call, which says). */
static int on_gpu(PyObject *t, const char *name, int *dev)
{
    PyObject *v = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!v) return 0;
    const long d = PyLong_AsLong(v);
    Py_DECREF(v);
    if (d == -1 && PyErr_Occurred()) return 0;
    if (d < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        return 0;
    }
    if (*dev >= 0 && d != *dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the tensors before it on cuda:%d", name, d, *dev);
        return 0;
    }
    *dev = (int)d;
    return 1;
}

static int contiguous(PyObject *t)
{
    PyObject *v = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!v) return -1;
    const int yes = v == Py_True;
    Py_DECREF(v);
    return yes;
}

/* A tuple of integers (shape, stride()): its length, its first `most` values; -1 on an error. */
static Py_ssize_t numbers(PyObject *tuple, int64_t *v, int most)
{
    if (!tuple) return -1;
    Py_ssize_t n = -1;
    if (PyTuple_Check(tuple)) {
        n = PyTuple_GET_SIZE(tuple);
        for (Py_ssize_t i = 0; i < n && i < most; ++i) {
            v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
            if (v[i] == -1 && PyErr_Occurred()) n = -1;
        }
    } else {
        PyErr_SetString(PyExc_TypeError, "a tensor's shape and strides must be tuples");
    }
    Py_DECREF(tuple);
    return n;
}

static Py_ssize_t shape_of(PyObject *t, int64_t *v, int most) { return numbers(PyObject_GetAttr(t, s_shape), v, most); }
static Py_ssize_t stride_of(PyObject *t, int64_t *v, int most) { return numbers(PyObject_CallMethodNoArgs(t, s_stride), v, most); }

static int address_of(PyObject *t, void **p)
{
    PyObject *v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return 0;
    *p = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

static void bad_shape(PyObject *t, const char *name, const char *want)
{
    if (PyErr_Occurred()) return;
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    PyErr_Format(PyExc_ValueError, "%s must be %s, got %S", name, want, shape ? shape : Py_None);
    Py_XDECREF(shape);
}

/* ---- arguments */

typedef struct {
    void *p;
    int64_t n, h, d, st, sh;
    int code;
} Rows;

/* A [tokens, heads, dim] tensor; heads, dim, tokens >= 0 are what it must have. */
static int rows(PyObject *t, const char *name, int64_t tokens, int64_t heads, int64_t dim, int *dev, Rows *r)
{
    int64_t v[3];
    if (!is_tensor(t, name)) return 0;
    PyObject *dtype = dtype_of(t);
    if (!dtype) return 0;
    if ((r->code = dtype_code(dtype)) < 0) {
        PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16, got %S", name, dtype);
        return 0;
    }
    if (!on_gpu(t, name, dev)) return 0;
    if (shape_of(t, v, 3) != 3 || (tokens >= 0 && v[0] != tokens) || (heads >= 0 && v[1] != heads) || (dim >= 0 && v[2] != dim)) {
        char want[96];
        if (tokens < 0 && heads < 0 && dim < 0) snprintf(want, sizeof want, "[tokens, heads, dim]");
        else snprintf(want, sizeof want, "[%lld, %lld, %lld] (-1: any)", (long long)tokens, (long long)heads, (long long)dim);
        bad_shape(t, name, want);
        return 0;
    }
    r->n = v[0], r->h = v[1], r->d = v[2];
    if (stride_of(t, v, 3) != 3) return 0;
    if (v[2] != 1 && r->d > 1) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous in its last dimension", name);
        return 0;
    }
    r->st = v[0], r->sh = v[1];
    return address_of(t, &r->p);
}

/* A contiguous device array of n values of a dtype. */
static int array(PyObject *t, const char *name, PyObject *want, int64_t n, int *dev, void **p)
{
    int64_t v[1];
    if (!is_tensor(t, name)) return 0;
    PyObject *dtype = dtype_of(t);
    if (!dtype) return 0;
    if (dtype != want) {
        PyErr_Format(PyExc_TypeError, "%s must have dtype %S, got %S", name, want, dtype);
        return 0;
    }
    if (!on_gpu(t, name, dev)) return 0;
    if (shape_of(t, v, 1) != 1 || v[0] != n || contiguous(t) != 1) {
        char text[64];
        snprintf(text, sizeof text, "a contiguous array of %lld", (long long)n);
        bad_shape(t, name, text);
        return 0;
    }
    return address_of(t, p);
}

static int array_or_none(PyObject *t, const char *name, PyObject *want, int64_t n, int *dev, void **p)
{
    *p = NULL;
    return t == Py_None || array(t, name, want, n, dev, p);
}

/* A rotary table or None. */
static int turn(PyObject *t, int64_t dim, int *dev, const float **p, int64_t *n, int64_t *rot)
{
    int64_t v[2];
    *p = NULL, *n = 0, *rot = 0;
    if (t == Py_None) return 1;
    if (!is_tensor(t, "table")) return 0;
    PyObject *dtype = dtype_of(t);
    if (!dtype) return 0;
    if (dtype != g_dtype[Q4K_F32]) {
        PyErr_Format(PyExc_TypeError, "table must have dtype %S, got %S", g_dtype[Q4K_F32], dtype);
        return 0;
    }
    if (!on_gpu(t, "table", dev)) return 0;
    if (shape_of(t, v, 2) != 2 || contiguous(t) != 1) {
        bad_shape(t, "table", "a contiguous [positions, rot] tensor");
        return 0;
    }
    if (v[1] % 2 || v[1] > dim) {
        PyErr_Format(PyExc_ValueError, "table turns %lld of %lld elements of a head", (long long)v[1], (long long)dim);
        return 0;
    }
    void *a;
    if (!address_of(t, &a)) return 0;
    *p = (const float *)a, *n = v[0], *rot = v[1];
    return 1;
}

/* Type code of a cache's dtype (16 bits, or 8), -1 for another one. */
static int cache_code(PyObject *dtype, int bits8)
{
    if (bits8) return dtype == g_int8 ? Q4K_I8 : dtype == g_e4m3 ? Q4K_E4M3 : -1;
    const int code = dtype_code(dtype);
    return code < Q4K_F16 ? -1 : code;
}

/* k_cache, v_cache at t, page_table, seq_start, kv_len at x. */
static int cache_parts(PyObject *const *t, PyObject *const *x, int64_t tokens, int bits8, int *dev, q4k_paged_cache *c)
{
    int64_t v[4], w[4];
    static const char *names[2] = {"k_cache", "v_cache"};
    int code[2];
    memset(c, 0, sizeof *c);
    for (int i = 0; i < 2; ++i) {
        if (!is_tensor(t[i], names[i])) return 0;
        PyObject *dtype = dtype_of(t[i]);
        if (!dtype) return 0;
        code[i] = cache_code(dtype, bits8);
        if (code[i] < 0 || code[i] != code[0]) {
            PyErr_Format(PyExc_TypeError, "%s must be %s, both caches the same, got %S", names[i],
                         bits8 ? "int8 or float8_e4m3fn" : "bfloat16 or float16", dtype);
            return 0;
        }
        if (!on_gpu(t[i], names[i], dev)) return 0;
    }
    if (shape_of(t[0], v, 4) != 4) {
        bad_shape(t[0], "k_cache", "[pages, page size, heads, dim]");
        return 0;
    }
    if (shape_of(t[1], w, 4) != 4 || memcmp(v, w, sizeof v)) {
        bad_shape(t[1], "v_cache", "of k_cache's shape");
        return 0;
    }
    c->pages = v[0], c->page_size = v[1], c->heads = v[2], c->dim = v[3], c->type = code[0];
    if (stride_of(t[0], v, 4) != 4 || stride_of(t[1], w, 4) != 4) return 0;
    if ((v[3] != 1 || w[3] != 1) && c->dim > 1) {
        PyErr_SetString(PyExc_ValueError, "k_cache and v_cache must be contiguous in their last dimension");
        return 0;
    }
    c->k_page_stride = v[0], c->k_slot_stride = v[1], c->k_head_stride = v[2];
    c->v_page_stride = w[0], c->v_slot_stride = w[1], c->v_head_stride = w[2];
    if (!is_tensor(x[0], "page_table")) return 0;
    PyObject *dtype = dtype_of(x[0]);
    if (!dtype) return 0;
    if (dtype != g_int32) {
        PyErr_Format(PyExc_TypeError, "page_table must have dtype %S, got %S", g_int32, dtype);
        return 0;
    }
    if (!on_gpu(x[0], "page_table", dev)) return 0;
    if (shape_of(x[0], v, 2) != 2) {
        bad_shape(x[0], "page_table", "[sequences, pages]");
        return 0;
    }
    if (stride_of(x[0], w, 2) != 2) return 0;
    if (w[1] != 1 && v[1] > 1) {
        PyErr_SetString(PyExc_ValueError, "page_table must be contiguous in its last dimension");
        return 0;
    }
    c->batch = v[0], c->max_pages = v[1], c->page_table_stride = w[0], c->tokens = tokens;
    return address_of(t[0], &c->k) && address_of(t[1], &c->v) && address_of(x[0], (void **)&c->page_table) &&
           array(x[1], "seq_start", g_int32, c->batch + 1, dev, (void **)&c->seq_start) &&
           array(x[2], "kv_len", g_int32, c->batch, dev, (void **)&c->kv_len);
}

static int cache(PyObject *const *t, int64_t tokens, int *dev, q4k_paged_cache *c)
{
    return cache_parts(t, t + 2, tokens, 0, dev, c);
}

/* k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len. */
static int cache8(PyObject *const *t, int64_t tokens, int *dev, q4k_paged_cache8 *c)
{
    static const char *names[2] = {"k_scale", "v_scale"};
    int64_t v[3], w[2][3], blocks = 0;
    memset(c, 0, sizeof *c);
    if (!cache_parts(t, t + 4, tokens, 1, dev, &c->cache)) return 0;
    for (int i = 0; i < 2; ++i) {
        PyObject *s = t[2 + i];
        if (!is_tensor(s, names[i])) return 0;
        PyObject *dtype = dtype_of(s);
        if (!dtype) return 0;
        if (dtype != g_dtype[Q4K_F32]) {
            PyErr_Format(PyExc_TypeError, "%s must have dtype %S, got %S", names[i], g_dtype[Q4K_F32], dtype);
            return 0;
        }
        if (!on_gpu(s, names[i], dev)) return 0;
        if (shape_of(s, v, 3) != 3 || v[0] != c->cache.pages || v[2] != c->cache.heads || v[1] < 1 || (i && v[1] != blocks) ||
            c->cache.page_size % v[1]) {
            bad_shape(s, names[i], "[pages, blocks of a page, heads], the same for keys and values");
            return 0;
        }
        blocks = v[1];
        if (stride_of(s, w[i], 3) != 3 || !address_of(s, i ? (void **)&c->v_scale : (void **)&c->k_scale)) return 0;
    }
    c->block = c->cache.page_size / blocks;
    if (c->block < 1 || c->block > 128 || (c->block & (c->block - 1))) {
        PyErr_Format(PyExc_ValueError, "a block of %lld tokens: a power of two up to 128 is wanted", (long long)c->block);
        return 0;
    }
    c->k_scale_page_stride = w[0][0], c->k_scale_block_stride = w[0][1], c->k_scale_head_stride = w[0][2];
    c->v_scale_page_stride = w[1][0], c->v_scale_block_stride = w[1][1], c->v_scale_head_stride = w[1][2];
    return 1;
}

/* A head norm's weight, fp32 [dim] or [heads, dim], or None. */
static int weight(PyObject *t, const char *name, int64_t heads, int64_t dim, int *dev, const float **p, int64_t *stride)
{
    int64_t v[2], w[2];
    *p = NULL, *stride = 0;
    if (t == Py_None) return 1;
    if (!is_tensor(t, name)) return 0;
    PyObject *dtype = dtype_of(t);
    if (!dtype) return 0;
    if (dtype != g_dtype[Q4K_F32]) {
        PyErr_Format(PyExc_TypeError, "%s must have dtype %S, got %S", name, g_dtype[Q4K_F32], dtype);
        return 0;
    }
    if (!on_gpu(t, name, dev)) return 0;
    const Py_ssize_t n = shape_of(t, v, 2);
    if (n < 1 || n > 2 || v[n - 1] != dim || (n == 2 && v[0] != heads)) {
        char want[96];
        snprintf(want, sizeof want, "[%lld] or [%lld, %lld]", (long long)dim, (long long)heads, (long long)dim);
        bad_shape(t, name, want);
        return 0;
    }
    if (stride_of(t, w, 2) != n) return 0;
    if (w[n - 1] != 1 && dim > 1) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous in its last dimension", name);
        return 0;
    }
    *stride = n == 2 ? w[0] : 0;
    void *a;
    if (!address_of(t, &a)) return 0;
    *p = (const float *)a;
    return 1;
}

static int epsilon(PyObject *v, float *eps)
{
    const double e = PyFloat_AsDouble(v);
    if (e == -1.0 && PyErr_Occurred()) return 0;
    if (!(e >= 0.0 && e <= 3e38)) {
        PyErr_SetString(PyExc_ValueError, "eps must be finite and not negative");
        return 0;
    }
    *eps = (float)e;
    return 1;
}

/* The handle of the call's stream: the given one's, or the current one of the tensors' device, which has to be
 * the current device (the library launches there). */
static int stream_of(PyObject *stream, int dev, void **s)
{
    PyObject *v = PyObject_CallNoArgs(g_device);
    if (!v) return 0;
    const long now = PyLong_AsLong(v);
    Py_DECREF(v);
    if (now == -1 && PyErr_Occurred()) return 0;
    if (now != dev) {
        PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%d, the current device is cuda:%ld", dev, now);
        return 0;
    }
    if (stream != Py_None) {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        PyObject *index = PyLong_FromLong(dev);
        if (!index) return 0;
        v = PyObject_CallOneArg(g_stream_of, index);
        Py_DECREF(index);
    }
    if (!v) return 0;
    *s = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return !PyErr_Occurred();
}

/* `out` checked against the wanted rows and dtype (None: any), or a new tensor like x of that dtype (None: x's)
 * of the call's stream (the current one, or `stream`).  A new reference, NULL on an error. */
static PyObject *output(PyObject *out, const char *name, PyObject *x, const Rows *like, PyObject *dtype, PyObject *stream, int *dev,
                        Rows *r)
{
    if (out != Py_None) {
        if (!rows(out, name, like->n, like->h, like->d, dev, r)) return NULL;
        if (dtype != Py_None && dtype_of(out) != dtype) {
            PyErr_Format(PyExc_TypeError, "%s must have dtype %S, got %S", name, dtype, dtype_of(out));
            return NULL;
        }
        Py_INCREF(out);
        return out;
    }
    const int code = dtype == Py_None ? like->code : dtype_code(dtype);
    if (code < 0) {
        PyErr_Format(PyExc_TypeError, "%s must be float32, float16 or bfloat16, got %S", name, dtype);
        return NULL;
    }
    PyObject *t = NULL;
    if (stream == Py_None && code == like->code && like->sh == like->d && like->st == like->h * like->d) {
        t = PyObject_CallOneArg(g_empty_like, x);
    } else {
        PyObject *device = PyObject_GetAttr(x, s_device);
        PyObject *shape = Py_BuildValue("(LLL)", (long long)like->n, (long long)like->h, (long long)like->d);
        if (device && shape) {
            if (stream == Py_None) {
                PyObject *args[3] = {shape, g_dtype[code], device};
                t = PyObject_Vectorcall(g_empty, args, 1, k_dtype_device);
            } else {
                PyObject *args[4] = {stream, shape, g_dtype[code], device};
                t = PyObject_Vectorcall(g_new_on, args, 4, NULL);
            }
        }
        Py_XDECREF(shape);
        Py_XDECREF(device);
    }
    if (!t) return NULL;
    r->n = like->n, r->h = like->h, r->d = like->d, r->sh = like->d, r->st = like->h * like->d, r->code = code;
    if (!address_of(t, &r->p)) {
        Py_DECREF(t);
        return NULL;
    }
    return t;
}

/* The result of a call: `out` (its reference), or the error that its status raises. */
static PyObject *result(const char *fn, q4k_status st, PyObject *out)
{
    if (st == Q4K_OK) return out;
    Py_XDECREF(out);
    PyObject *v = PyObject_CallFunction(g_raise, "si", fn, (int)st);
    Py_XDECREF(v);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed: status %d", fn, (int)st);
    return NULL;
}

static int wants(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return 0;
}

/* ---- the calls (positional, as _attention.py passes them) */

/* x, pos, table, y, interleaved, out_dtype, stream, pdl */
static PyObject *rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Rows x, y;
    q4k_rope_args r;
    void *stream;
    int dev = -1;
    memset(&r, 0, sizeof r);
    if (!wants(n, 8) || !rows(a[0], "x", -1, -1, -1, &dev, &x) || !turn(a[2], x.d, &dev, &r.table, &r.table_rows, &r.rot)) return NULL;
    if (r.rot && a[1] == Py_None) {
        PyErr_SetString(PyExc_ValueError, "pos is needed with a table");
        return NULL;
    }
    if (!array_or_none(a[1], "pos", g_int32, x.n, &dev, (void **)&r.pos) || !stream_of(a[6], dev, &stream)) return NULL;
    const int inter = PyObject_IsTrue(a[4]), pdl = PyObject_IsTrue(a[7]);
    if (inter < 0 || pdl < 0) return NULL;
    PyObject *out = output(a[3], "y", a[0], &x, a[5], a[6], &dev, &y);
    if (!out) return NULL;
    r.x = x.p, r.y = y.p;
    r.tokens = x.n, r.heads = x.h, r.dim = x.d;
    r.x_token_stride = x.st, r.x_head_stride = x.sh, r.y_token_stride = y.st, r.y_head_stride = y.sh;
    r.x_type = x.code, r.y_type = y.code, r.interleaved = inter, r.flags = pdl ? Q4K_FLAG_PDL : 0;
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = g_rope(&r, stream);
    Py_END_ALLOW_THREADS return result("q4k_rope", st, out);
}

/* k, v, k_cache, v_cache, page_table, seq_start, kv_len, table, interleaved, pos, q, q_out, q_dtype, stream, pdl */
static PyObject *kv_append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Rows k, v, q, o;
    q4k_paged_cache c;
    q4k_append_args r;
    void *stream;
    int dev = -1;
    memset(&r, 0, sizeof r);
    if (!wants(n, 15) || !rows(a[0], "k", -1, -1, -1, &dev, &k) || !rows(a[1], "v", k.n, k.h, k.d, &dev, &v)) return NULL;
    if (v.code != k.code) {
        PyErr_SetString(PyExc_TypeError, "k and v must have the same dtype");
        return NULL;
    }
    if (!cache(a + 2, k.n, &dev, &c)) return NULL;
    if (c.heads != k.h || c.dim != k.d) {
        PyErr_Format(PyExc_ValueError, "the cache holds %lld heads of %lld, k and v %lld of %lld", (long long)c.heads,
                     (long long)c.dim, (long long)k.h, (long long)k.d);
        return NULL;
    }
    if (!turn(a[7], k.d, &dev, &r.table, &r.table_rows, &r.rot) || !array_or_none(a[9], "pos", g_int32, k.n, &dev, (void **)&r.pos) ||
        !stream_of(a[13], dev, &stream))
        return NULL;
    const int inter = PyObject_IsTrue(a[8]), pdl = PyObject_IsTrue(a[14]);
    if (inter < 0 || pdl < 0) return NULL;
    PyObject *out = NULL;
    if (a[10] != Py_None) {
        if (!rows(a[10], "q", k.n, -1, k.d, &dev, &q)) return NULL;
        out = output(a[11], "q_out", a[10], &q, a[12], a[13], &dev, &o);
        if (!out) return NULL;
        r.q = q.p, r.q_out = o.p, r.q_heads = q.h;
        r.q_token_stride = q.st, r.q_head_stride = q.sh, r.q_out_token_stride = o.st, r.q_out_head_stride = o.sh;
        r.q_type = q.code, r.q_out_type = o.code;
    } else {
        if (a[11] != Py_None) {
            PyErr_SetString(PyExc_ValueError, "q_out without q");
            return NULL;
        }
        out = Py_None;
        Py_INCREF(out);
    }
    r.k = k.p, r.v = v.p;
    r.k_token_stride = k.st, r.k_head_stride = k.sh, r.v_token_stride = v.st, r.v_head_stride = v.sh;
    r.kv_type = k.code, r.interleaved = inter, r.flags = pdl ? Q4K_FLAG_PDL : 0;
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = g_append(&c, &r, stream);
    Py_END_ALLOW_THREADS return result("q4k_kv_append", st, out);
}

/* q, k_cache, v_cache, page_table, seq_start, kv_len, out, scale, out_dtype, softcap, slopes, window, causal, prefix_len,
 * kv_start, lse, stream, flags, wait_limit_us */
static PyObject *attention(PyObject *const *a, Py_ssize_t n, int bits8)
{
    Rows q, o;
    q4k_paged_cache8 c8;
    q4k_paged_cache c;
    q4k_attention_args r;
    void *stream;
    int dev = -1;
    memset(&r, 0, sizeof r);
    if (!wants(n, 19 + 2 * bits8) || !rows(a[0], "q", -1, -1, -1, &dev, &q)) return NULL;
    if (bits8) {
        if (!cache8(a + 1, q.n, &dev, &c8)) return NULL;
        c = c8.cache;
    } else if (!cache(a + 1, q.n, &dev, &c)) {
        return NULL;
    }
    PyObject *const q_tensor = a[0];
    a += 2 * bits8;   /* (the scales' places) */
    if (c.dim != q.d || c.heads < 1 || q.h % c.heads) {
        PyErr_Format(PyExc_ValueError, "the cache holds %lld heads of %lld, q %lld of %lld", (long long)c.heads,
                     (long long)c.dim, (long long)q.h, (long long)q.d);
        return NULL;
    }
    const double scale = a[7] == Py_None ? 1.0 / sqrt((double)q.d) : PyFloat_AsDouble(a[7]), cap = PyFloat_AsDouble(a[9]);
    r.window = PyLong_AsLongLong(a[11]);
    const int causal = PyObject_IsTrue(a[12]);
    const unsigned long limit = PyLong_AsUnsignedLong(a[18]);
    r.flags = (uint32_t)PyLong_AsUnsignedLong(a[17]), r.wait_limit_us = (uint32_t)limit;
    if (PyErr_Occurred()) return NULL;
    if (limit > UINT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "wait_limit_us must be less than 2^32");
        return NULL;
    }
    if (!array_or_none(a[10], "slopes", g_dtype[Q4K_F32], q.h, &dev, (void **)&r.slopes) ||
        !array_or_none(a[13], "prefix_len", g_int32, c.batch, &dev, (void **)&r.prefix_len) ||
        !array_or_none(a[14], "kv_start", g_int32, q.n, &dev, (void **)&r.kv_start))
        return NULL;
    if (a[15] != Py_None) {
        int64_t v[2];
        if (!is_tensor(a[15], "lse")) return NULL;
        if (dtype_of(a[15]) != g_dtype[Q4K_F32]) {
            PyErr_SetString(PyExc_TypeError, "lse must be a float32 tensor");
            return NULL;
        }
        if (!on_gpu(a[15], "lse", &dev)) return NULL;
        if (shape_of(a[15], v, 2) != 2 || v[0] != q.n || v[1] != q.h || contiguous(a[15]) != 1) {
            bad_shape(a[15], "lse", "a contiguous [tokens, q heads] tensor");
            return NULL;
        }
        if (!address_of(a[15], (void **)&r.lse)) return NULL;
    }
    if (!stream_of(a[16], dev, &stream)) return NULL;
    PyObject *out = output(a[6], "out", q_tensor, &q, a[8], a[16], &dev, &o);
    if (!out) return NULL;
    r.q = q.p, r.out = o.p;
    r.q_token_stride = q.st, r.q_head_stride = q.sh, r.out_token_stride = o.st, r.out_head_stride = o.sh;
    r.q_heads = q.h, r.scale = (float)scale, r.softcap = (float)cap;
    r.q_type = q.code, r.out_type = o.code, r.causal = causal;
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = bits8 ? g_attention8(&c8, &r, stream) : g_attention(&c, &r, stream);
    Py_END_ALLOW_THREADS return result(bits8 ? "q4k_paged_attention8" : "q4k_paged_attention", st, out);
}

static PyObject *paged_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) { return attention(a, n, 0); }

/* The same with k_scale, v_scale behind the caches. */
static PyObject *paged_attention8(PyObject *self, PyObject *const *a, Py_ssize_t n) { return attention(a, n, 1); }

/* q, k, pos, table, q_weight, k_weight, q_out, k_out, eps, interleaved, out_dtype, stream, pdl */
static PyObject *norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Rows x, y;
    q4k_norm_rope_args r;
    void *stream;
    int dev = -1;
    memset(&r, 0, sizeof r);
    if (!wants(n, 13) || !rows(a[0], "q", -1, -1, -1, &dev, &x) || !turn(a[3], x.d, &dev, &r.table, &r.table_rows, &r.rot)) return NULL;
    if (r.rot && a[2] == Py_None) {
        PyErr_SetString(PyExc_ValueError, "pos is needed with a table");
        return NULL;
    }
    if (!array_or_none(a[2], "pos", g_int32, x.n, &dev, (void **)&r.pos) || !stream_of(a[11], dev, &stream) || !epsilon(a[8], &r.eps))
        return NULL;
    const int inter = PyObject_IsTrue(a[9]), pdl = PyObject_IsTrue(a[12]);
    if (inter < 0 || pdl < 0) return NULL;
    r.tokens = x.n, r.dim = x.d, r.interleaved = inter, r.flags = pdl ? Q4K_FLAG_PDL : 0;
    PyObject *out[2] = {NULL, NULL};
    q4k_heads *to[2] = {&r.q, &r.k};
    const int two = a[1] != Py_None;
    if (!two && (a[5] != Py_None || a[7] != Py_None)) {
        PyErr_SetString(PyExc_ValueError, "k_weight or k_out without k");
        return NULL;
    }
    for (int i = 0; i <= two; ++i) {
        q4k_heads *h = to[i];
        if ((i && !rows(a[1], "k", r.tokens, -1, r.dim, &dev, &x)) ||
            !weight(a[4 + i], i ? "k_weight" : "q_weight", x.h, x.d, &dev, &h->weight, &h->weight_head_stride) ||
            !(out[i] = output(a[6 + i], i ? "k_out" : "q_out", a[i], &x, a[10], a[11], &dev, &y))) {
            Py_XDECREF(out[0]);
            return NULL;
        }
        h->x = x.p, h->y = y.p, h->heads = x.h, h->x_type = x.code, h->y_type = y.code;
        h->x_token_stride = x.st, h->x_head_stride = x.sh, h->y_token_stride = y.st, h->y_head_stride = y.sh;
    }
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = g_norm_rope(&r, stream);
    Py_END_ALLOW_THREADS
    if (!two) {
        out[1] = Py_None;
        Py_INCREF(out[1]);
    }
    PyObject *both = PyTuple_Pack(2, out[0], out[1]);
    Py_DECREF(out[0]);
    Py_DECREF(out[1]);
    return both ? result("q4k_norm_rope", st, both) : NULL;
}

/* k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, table, interleaved, pos, q, q_out, q_dtype, q_weight,
 * k_weight, eps, stream, pdl */
static PyObject *kv_append8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Rows k, v, q, o;
    q4k_paged_cache8 c;
    q4k_append8_args r8;
    q4k_append_args *r = &r8.a;
    void *stream;
    int dev = -1;
    memset(&r8, 0, sizeof r8);
    if (!wants(n, 20) || !rows(a[0], "k", -1, -1, -1, &dev, &k) || !rows(a[1], "v", k.n, k.h, k.d, &dev, &v)) return NULL;
    if (v.code != k.code) {
        PyErr_SetString(PyExc_TypeError, "k and v must have the same dtype");
        return NULL;
    }
    if (!cache8(a + 2, k.n, &dev, &c)) return NULL;
    if (c.cache.heads != k.h || c.cache.dim != k.d) {
        PyErr_Format(PyExc_ValueError, "the cache holds %lld heads of %lld, k and v %lld of %lld", (long long)c.cache.heads,
                     (long long)c.cache.dim, (long long)k.h, (long long)k.d);
        return NULL;
    }
    if (!turn(a[9], k.d, &dev, &r->table, &r->table_rows, &r->rot) || !array_or_none(a[11], "pos", g_int32, k.n, &dev, (void **)&r->pos) ||
        !weight(a[16], "k_weight", k.h, k.d, &dev, &r8.k_weight, &r8.k_weight_head_stride) || !epsilon(a[17], &r8.eps) ||
        !stream_of(a[18], dev, &stream))
        return NULL;
    const int inter = PyObject_IsTrue(a[10]), pdl = PyObject_IsTrue(a[19]);
    if (inter < 0 || pdl < 0) return NULL;
    PyObject *out = NULL;
    if (a[12] != Py_None) {
        if (!rows(a[12], "q", k.n, -1, k.d, &dev, &q) ||
            !weight(a[15], "q_weight", q.h, q.d, &dev, &r8.q_weight, &r8.q_weight_head_stride))
            return NULL;
        out = output(a[13], "q_out", a[12], &q, a[14], a[18], &dev, &o);
        if (!out) return NULL;
        r->q = q.p, r->q_out = o.p, r->q_heads = q.h;
        r->q_token_stride = q.st, r->q_head_stride = q.sh, r->q_out_token_stride = o.st, r->q_out_head_stride = o.sh;
        r->q_type = q.code, r->q_out_type = o.code;
    } else {
        if (a[13] != Py_None || a[15] != Py_None) {
            PyErr_SetString(PyExc_ValueError, "q_out or q_weight without q");
            return NULL;
        }
        out = Py_None;
        Py_INCREF(out);
    }
    r->k = k.p, r->v = v.p;
    r->k_token_stride = k.st, r->k_head_stride = k.sh, r->v_token_stride = v.st, r->v_head_stride = v.sh;
    r->kv_type = k.code, r->interleaved = inter, r->flags = pdl ? Q4K_FLAG_PDL : 0;
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = g_append8(&c, &r8, stream);
    Py_END_ALLOW_THREADS return result("q4k_kv_append8", st, out);
}

/* k_cache, v_cache, k_scale, v_scale, page_table, seq_start, kv_len, tokens, k, v, dtype, stream, pdl */
static PyObject *kv_read8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Rows like, y[2];
    q4k_paged_cache8 c;
    q4k_read8_args r;
    void *stream;
    int dev = -1;
    memset(&r, 0, sizeof r);
    if (!wants(n, 13)) return NULL;
    const int64_t tokens = PyLong_AsLongLong(a[7]);
    if (PyErr_Occurred()) return NULL;
    if (tokens < 0) {
        PyErr_SetString(PyExc_ValueError, "tokens must not be negative");
        return NULL;
    }
    if (!cache8(a, tokens, &dev, &c) || !stream_of(a[11], dev, &stream)) return NULL;
    const int pdl = PyObject_IsTrue(a[12]);
    if (pdl < 0) return NULL;
    /* (a code of no row type: a new output is made with its own) */
    like.n = tokens, like.h = c.cache.heads, like.d = c.cache.dim, like.st = like.sh = 0, like.code = -1;
    PyObject *out[2] = {NULL, NULL};
    for (int i = 0; i < 2; ++i)
        if (!(out[i] = output(a[8 + i], i ? "v" : "k", a[i], &like, a[10], a[11], &dev, &y[i]))) {
            Py_XDECREF(out[0]);
            return NULL;
        }
    if (y[0].code != y[1].code) {
        PyErr_SetString(PyExc_TypeError, "k and v must have the same dtype");
        Py_DECREF(out[0]);
        Py_DECREF(out[1]);
        return NULL;
    }
    r.k = y[0].p, r.v = y[1].p, r.type = y[0].code, r.flags = pdl ? Q4K_FLAG_PDL : 0;
    r.k_token_stride = y[0].st, r.k_head_stride = y[0].sh, r.v_token_stride = y[1].st, r.v_head_stride = y[1].sh;
    q4k_status st;
    Py_BEGIN_ALLOW_THREADS st = g_read8(&c, &r, stream);
    Py_END_ALLOW_THREADS
    PyObject *both = PyTuple_Pack(2, out[0], out[1]);
    Py_DECREF(out[0]);
    Py_DECREF(out[1]);
    return both ? result("q4k_kv_read8", st, both) : NULL;
}

/* int8, float8_e4m3fn, and the addresses of q4k_norm_rope, q4k_kv_append8, q4k_kv_read8, q4k_paged_attention8 (after setup). */
static PyObject *setup8(PyObject *self, PyObject *args)
{
    PyObject *o[2];
    unsigned long long f[4];
    if (!PyArg_ParseTuple(args, "OOKKKK", &o[0], &o[1], &f[0], &f[1], &f[2], &f[3])) return NULL;
    for (int i = 0; i < 2; ++i) Py_INCREF(o[i]);   /* kept */
    g_int8 = o[0], g_e4m3 = o[1];
    g_norm_rope = (norm_rope_fn)(uintptr_t)f[0], g_append8 = (append8_fn)(uintptr_t)f[1], g_read8 = (read8_fn)(uintptr_t)f[2];
    g_attention8 = (attention8_fn)(uintptr_t)f[3];
    Py_RETURN_NONE;
}

/* Tensor, float32, float16, bfloat16, int32, empty, empty_like, new_on(stream, shape, dtype, device), current device, current stream's handle of a device, raise(fn, status),
 * and the addresses of q4k_rope, q4k_kv_append, q4k_paged_attention. */
static PyObject *setup(PyObject *self, PyObject *args)
{
    PyObject *o[11];
    unsigned long long f[3];
    if (!PyArg_ParseTuple(args, "OOOOOOOOOOOKKK", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &o[6], &o[7], &o[8], &o[9], &o[10], &f[0],
                          &f[1], &f[2]))
        return NULL;
    if (!PyType_Check(o[0])) {
        PyErr_SetString(PyExc_TypeError, "the Tensor class is wanted first");
        return NULL;
    }
    for (int i = 0; i < 11; ++i) Py_INCREF(o[i]);   /* kept */
    g_tensor = o[0], g_dtype[Q4K_F32] = o[1], g_dtype[Q4K_F16] = o[2], g_dtype[Q4K_BF16] = o[3], g_int32 = o[4];
    g_empty = o[5], g_empty_like = o[6], g_new_on = o[7], g_device = o[8], g_stream_of = o[9], g_raise = o[10];
    g_rope = (rope_fn)(uintptr_t)f[0], g_append = (append_fn)(uintptr_t)f[1], g_attention = (attention_fn)(uintptr_t)f[2];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "What the calls need of torch and of the library."},
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, "q4k_rope"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, "q4k_kv_append"},
    {"setup8", setup8, METH_VARARGS, "The same of an 8-bit cache's calls."},
    {"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, "q4k_norm_rope"},
    {"kv_append8", (PyCFunction)(void (*)(void))kv_append8, METH_FASTCALL, "q4k_kv_append8"},
    {"kv_read8", (PyCFunction)(void (*)(void))kv_read8, METH_FASTCALL, "q4k_kv_read8"},
    {"paged_attention8", (PyCFunction)(void (*)(void))paged_attention8, METH_FASTCALL, "q4k_paged_attention8"},
    {"paged_attention", (PyCFunction)(void (*)(void))paged_attention, METH_FASTCALL, "q4k_paged_attention"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument marshalling of the attention operators.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    struct {
        PyObject **to;
        const char *text;
    } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"},
                 {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"},
                 {&s_device, "device"}, {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].text))) return NULL;
    k_dtype_device = PyTuple_Pack(2, s_dtype, s_device);
    if (!k_dtype_device) return NULL;
    return PyModule_Create(&module);
}
