/* The binding's native half for the calls that run per layer and step
 * (kv_page_plan, kv_rope_store, kv_attention_bf16, norm_gate_residual,
 * moe_route_topk, fp8_quantize, swiglu_fp8_rows, fp8_gemm, fp8_moe): it reads address, type, shape and strides off the tensors,
 * checks that they fit one another, and calls the C ABI.  Done in Python and
 * through ctypes the same took 5 to 9 us a call on the host, more than the
 * kernels of a decoded token take on the device.
 *
 * Tensors come as Python objects and are read through their attributes, so
 * this file needs Python's headers alone.  The library's functions come as
 * addresses (setup()).  A refused argument raises ValueError or TypeError;
 * otherwise the call's status is returned. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <math.h>
#include <stdint.h>

#include "../../include/q2k.h"

static PyObject *n_get_device, *n_dtype, *n_data_ptr, *n_shape, *n_stride;
static PyObject *t_f32, *t_bf16, *t_i32, *t_i64, *t_u8;
static PyObject* current_device;  /* a callable */

static int (*f_plan)(const int32_t*, const int32_t*, int64_t, int64_t, const int32_t*, int64_t, const int32_t*, int32_t*,
                     int64_t, int64_t, int32_t*, int32_t*, int32_t*, int32_t*, int32_t*, int64_t, int32_t*, int32_t*,
                     q2k_stream_t);
static int (*f_rope)(const void*, int64_t, const void*, int64_t, const void*, int64_t, int, int64_t, int64_t, int64_t,
                     int64_t, const int32_t*, int64_t, const int32_t*, const float*, int64_t, int, const int32_t*,
                     uint16_t*, int64_t, uint16_t*, uint16_t*, int64_t, int64_t, int64_t, int32_t*, q2k_stream_t);
static int (*f_attn)(const uint16_t*, int64_t, int64_t, int64_t, int64_t, int64_t, const uint16_t*, const uint16_t*,
                     int64_t, int64_t, int64_t, const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*,
                     int64_t, float, int64_t, uint16_t*, int64_t, float*, void*, size_t, q2k_stream_t);
static size_t (*f_attn_bytes)(int64_t, int64_t, int64_t, int64_t);
static int (*f_norm)(const void*, int, int64_t, const float*, const void*, int64_t, const void*, int, int64_t, float,
                     const float*, float, int64_t, int64_t, void*, int64_t, uint16_t*, int64_t, void*, q2k_stream_t);
static int (*f_route)(const void*, int, int64_t, int64_t, int64_t, const float*, int, int64_t, int64_t, int64_t, int,
                      float, int32_t*, float*, const int64_t*, int64_t*, q2k_stream_t);
static PyObject* t_e4m3;
static int (*f_quantize)(const void*, int, int64_t, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t,
                         q2k_stream_t);
static int (*f_swiglu)(const void*, int, int64_t, int64_t, int64_t, uint8_t*, int64_t, float*, int64_t, q2k_stream_t);
static int (*f_gemm)(const uint8_t*, int64_t, int64_t, int64_t, const float*, int64_t, const uint8_t*, int64_t,
                     const float*, void*, int, int64_t, q2k_stream_t);
static size_t (*f_moe_bytes)(int64_t, int64_t, int64_t, int64_t);
static int (*f_moe)(const uint16_t*, int64_t, int64_t, int64_t, const int32_t*, const float*, int64_t, int64_t,
                    const uint8_t*, const float*, const uint8_t*, const float*, int64_t, void*, int, int64_t, void*,
                    size_t, q2k_stream_t);

/* ---- tensors ---------------------------------------------------------------- */

#define MAX_DIMS 4

typedef struct {
    void* p;  /* NULL for None */
    int dims;
    int64_t size[MAX_DIMS], stride[MAX_DIMS], count;
    PyObject* dtype;  /* borrowed from the tensor's type object: the dtypes are singletons */
} Tensor;

static int read_ints(PyObject* seq, int64_t* to, const char* name)
{
    if (!seq)
        return -1;
    if (!PyTuple_Check(seq) || PyTuple_GET_SIZE(seq) > MAX_DIMS) {
        Py_DECREF(seq);
        PyErr_Format(PyExc_ValueError, "%s has too many dimensions", name);
        return -1;
    }
    const int n = (int)PyTuple_GET_SIZE(seq);
    for (int i = 0; i < n; ++i) {
        to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(seq, i));
        if (to[i] == -1 && PyErr_Occurred()) {
            Py_DECREF(seq);
            return -1;
        }
    }
    Py_DECREF(seq);
    return n;
}

/* The device that the kernels of the call at hand run on, asked once a call. */
static _Thread_local long launch_device;

static void begin_call(void) { launch_device = -1; }

static int on_launch_device(long device, const char* name)
{
    if (device < 0) {
        PyErr_Format(PyExc_ValueError, "tensors must be on a CUDA device (%s is not)", name);
        return -1;
    }
    if (launch_device < 0) {
        PyObject* v = PyObject_CallNoArgs(current_device);
        if (!v)
            return -1;
        launch_device = PyLong_AsLong(v);
        Py_DECREF(v);
        if (launch_device < 0) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_RuntimeError, "no current CUDA device");
            return -1;
        }
    }
    if (device != launch_device) {
        PyErr_Format(PyExc_ValueError, "tensors must be on the current CUDA device, %ld (%s is on %ld)", launch_device, name,
                     device);
        return -1;
    }
    return 0;
}

/* A tensor of the current CUDA device and the given type (any, where type is NULL); None gives p = NULL when it may. */
static int read_tensor(PyObject* t, PyObject* type, const char* name, int may_be_none, Tensor* x)
{
    x->p = NULL;
    x->dims = 0;
    x->count = 0;
    x->dtype = NULL;
    if (t == Py_None) {
        if (may_be_none)
            return 0;
        PyErr_Format(PyExc_ValueError, "%s is required", name);
        return -1;
    }
    PyObject* v = PyObject_CallMethodNoArgs(t, n_get_device);  /* -1 on the host */
    if (!v)
        return -1;
    const long device = PyLong_AsLong(v);
    Py_DECREF(v);
    if ((device == -1 && PyErr_Occurred()) || on_launch_device(device, name))
        return -1;
    if (!(v = PyObject_GetAttr(t, n_dtype)))
        return -1;
    x->dtype = v;
    Py_DECREF(v);
    if (type && x->dtype != type) {
        PyErr_Format(PyExc_TypeError, "%s must be %S, not %S", name, type, x->dtype);
        return -1;
    }
    if ((x->dims = read_ints(PyObject_GetAttr(t, n_shape), x->size, name)) < 0 ||
        read_ints(PyObject_CallMethodNoArgs(t, n_stride), x->stride, name) < 0)
        return -1;
    x->count = 1;
    for (int i = 0; i < x->dims; ++i)
        x->count *= x->size[i];
    if (!(v = PyObject_CallMethodNoArgs(t, n_data_ptr)))
        return -1;
    x->p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return x->p || !PyErr_Occurred() ? 0 : -1;
}

static int dense(const Tensor* x, const char* name)
{
    int64_t want = 1;
    for (int i = x->dims - 1; i >= 0; --i) {
        if (x->size[i] != 1 && x->stride[i] != want && x->count) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            return -1;
        }
        want *= x->size[i];
    }
    return 0;
}

static int read_dense(PyObject* t, PyObject* type, const char* name, int may_be_none, Tensor* x)
{
    return read_tensor(t, type, name, may_be_none, x) || dense(x, name) ? -1 : 0;
}

static int fail(const char* what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

static int type_of(const Tensor* x, const char* name)
{
    if (x->dtype == t_f32)
        return Q2K_F32;
    if (x->dtype == t_bf16)
        return Q2K_BF16;
    PyErr_Format(PyExc_TypeError, "%s must be fp32 or bf16, not %S", name, x->dtype);
    return -1;
}

/* [T, H, D] whose heads of a token lie back to back: the stride between tokens. */
static int heads(const Tensor* x, const char* name, int64_t* ld)
{
    if (x->dims != 3 || (x->size[2] > 1 && x->stride[2] != 1) || (x->size[1] > 1 && x->stride[1] != x->size[2])) {
        PyErr_Format(PyExc_ValueError, "%s must be [T, H, D] with the heads of a token back to back", name);
        return -1;
    }
    const int64_t row = x->size[1] * x->size[2];
    *ld = x->size[0] > 1 || x->stride[0] > row ? x->stride[0] : row;
    return 0;
}

/* [T, dim] with dense rows: the stride between them. */
static int rows(const Tensor* x, int64_t T, int64_t dim, const char* name, int64_t* ld)
{
    if (x->dims != 2 || x->size[0] != T || x->size[1] != dim || (dim > 1 && x->stride[1] != 1)) {
        PyErr_Format(PyExc_ValueError, "%s must be [T, dim] with dense rows", name);
        return -1;
    }
    *ld = T > 1 || x->stride[0] > dim ? x->stride[0] : dim;
    return 0;
}

/* [n_pages, Hkv, page_size, D] twice, pages dense, the pages themselves at any equal stride. */
static int cache(const Tensor* k, const Tensor* v, int64_t* page_stride)
{
    if (k->dims != 4 || v->dims != 4)
        return fail("the caches must be [n_pages, Hkv, page_size, D]");
    for (int i = 0; i < 4; ++i)
        if (k->size[i] != v->size[i] || (k->stride[i] != v->stride[i] && k->size[i] > 1))
            return fail("k_cache and v_cache must have one shape and one set of strides");
    int64_t want = 1;
    for (int i = 3; i >= 1; --i) {
        if (k->size[i] > 1 && k->stride[i] != want)
            return fail("a page of the cache must be contiguous [Hkv, page_size, D]");
        want *= k->size[i];
    }
    *page_stride = k->size[0] > 1 || k->stride[0] > want ? k->stride[0] : want;
    return 0;
}

static int want_args(Py_ssize_t got, Py_ssize_t n)
{
    if (got == n)
        return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", n, got);
    return -1;
}

static int64_t as_int(PyObject* o) { return PyLong_AsLongLong(o); }
static float as_float(PyObject* o) { return (float)PyFloat_AsDouble(o); }
static q2k_stream_t as_stream(PyObject* o) { return (q2k_stream_t)(uintptr_t)PyLong_AsUnsignedLongLong(o); }

static PyObject* status(int st) { return PyLong_FromLong(st); }

/* ---- the calls -------------------------------------------------------------- */

/* ctx_lens, new_lens, page_size, free_pages, free_head, block_table, max_tokens, outs, err_flag, stream;
 * outs: one int32 buffer for all six arrays in a row, or a tuple of six. */
static PyObject* py_plan(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor ctx, add, pool, head, table, err, o[6];
    static const char* const names[6] = {"cu_q", "seq_lens", "positions", "token_req", "slot_map", "free_head"};
    if (want_args(n, 10) || read_dense(a[0], t_i32, "ctx_lens", 0, &ctx) ||
        read_dense(a[1], t_i32, "new_lens", 0, &add) || read_dense(a[3], t_i32, "free_pages", 0, &pool) ||
        read_dense(a[4], t_i32, "free_head", 1, &head) || read_tensor(a[5], t_i32, "block_table", 0, &table) ||
        read_dense(a[8], t_i32, "err_flag", 1, &err))
        return NULL;
    const int64_t reqs = ctx.count, page = as_int(a[2]), max_tokens = as_int(a[6]);
    const int64_t want[6] = {reqs + 1, reqs, max_tokens, max_tokens, max_tokens, 1};
    int64_t ld = 0;
    if (PyErr_Occurred())
        return NULL;
    if (add.count != reqs || table.dims != 2 || table.size[0] != reqs) {
        fail("one ctx_len, new_len and row of block_table per request");
        return NULL;
    }
    if (rows(&table, reqs, table.size[1], "block_table", &ld))
        return NULL;
    if (PyTuple_Check(a[7])) {
        if (PyTuple_GET_SIZE(a[7]) != 6) {
            fail("out must be a PagePlan");
            return NULL;
        }
        for (int i = 0; i < 6; ++i) {
            if (read_dense(PyTuple_GET_ITEM(a[7], i), t_i32, names[i], 0, &o[i]))
                return NULL;
            if (o[i].count != want[i]) {
                fail("out does not fit n_req and max_tokens");
                return NULL;
            }
        }
    } else {
        Tensor all;
        if (read_dense(a[7], t_i32, "out", 0, &all))
            return NULL;
        if (all.count != 2 * reqs + 3 * max_tokens + 2) {
            fail("out does not fit n_req and max_tokens");
            return NULL;
        }
        int32_t* p = all.p;
        for (int i = 0; i < 6; ++i) {
            o[i].p = p;
            p += want[i];
        }
    }
    const q2k_stream_t stream = as_stream(a[9]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_plan(ctx.p, add.p, reqs, page, pool.p, pool.count, head.p, table.p, table.size[1], ld, o[0].p, o[1].p,
                         o[2].p, o[3].p, o[4].p, max_tokens, o[5].p, err.p, stream));
}

/* q, k, v, positions, inv_freq, slot_map, k_cache, v_cache, sections, interleaved, q_out, err_flag, stream */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor q, k, v, pos, freq, slots, kc, vc, out, err;
    if (want_args(n, 13) || read_tensor(a[1], NULL, "k", 0, &k))
        return NULL;
    const int type = type_of(&k, "k");
    int64_t ld_q = 0, ld_k, ld_v, ld_o = 0, page_stride;
    if (type < 0 || read_tensor(a[0], k.dtype, "q", 1, &q) || read_tensor(a[2], k.dtype, "v", 0, &v) ||
        read_dense(a[3], t_i32, "positions", 0, &pos) || read_dense(a[4], t_f32, "inv_freq", 0, &freq) ||
        read_dense(a[5], t_i32, "slot_map", 0, &slots) || read_tensor(a[6], t_bf16, "k_cache", 0, &kc) ||
        read_tensor(a[7], t_bf16, "v_cache", 0, &vc) || read_tensor(a[10], t_bf16, "q_out", 1, &out) ||
        read_dense(a[11], t_i32, "err_flag", 1, &err) || heads(&k, "k", &ld_k) || heads(&v, "v", &ld_v) ||
        cache(&kc, &vc, &page_stride))
        return NULL;
    const int has_q = a[0] != Py_None;
    if (has_q && (heads(&q, "q", &ld_q) || heads(&out, "q_out", &ld_o)))
        return NULL;
    const int64_t T = k.size[0], H = k.size[1], D = k.size[2], axes = pos.dims > 1 ? pos.size[0] : 1;
    if (v.size[0] != T || v.size[1] != H || v.size[2] != D || kc.size[1] != H || kc.size[3] != D || slots.count != T ||
        pos.count != axes * T) {
        fail("k, v, positions, slot_map and the cache do not fit one another");
        return NULL;
    }
    if (has_q && (q.size[0] != T || q.size[2] != D || out.size[0] != T || out.size[1] != q.size[1] || out.size[2] != D)) {
        fail("q, q_out and k do not fit one another");
        return NULL;
    }
    if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != axes || axes > 3) {
        fail("one section per axis, three at most");
        return NULL;
    }
    int32_t sections[3] = {0, 0, 0};
    for (int i = 0; i < axes; ++i)
        sections[i] = (int32_t)as_int(PyTuple_GET_ITEM(a[8], i));
    const int interleaved = PyObject_IsTrue(a[9]);
    const q2k_stream_t stream = as_stream(a[12]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_rope(q.p, ld_q, k.p, ld_k, v.p, ld_v, type, T, has_q ? q.size[1] : 0, H, D, pos.p, axes, sections,
                         freq.p, 2 * freq.count, interleaved, slots.p, out.p, ld_o, kc.p, vc.p, kc.size[0], kc.size[2],
                         page_stride, err.p, stream));
}

/* q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, window, out, lse, workspace, stream */
static PyObject* py_attn(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor q, kc, vc, table, cu, seq, out, lse, ws;
    int64_t ld_q, ld_o, ld_t = 0, page_stride;
    if (want_args(n, 12) || read_tensor(a[0], t_bf16, "q", 0, &q) || read_tensor(a[1], t_bf16, "k_cache", 0, &kc) ||
        read_tensor(a[2], t_bf16, "v_cache", 0, &vc) || read_tensor(a[3], t_i32, "block_table", 0, &table) ||
        read_dense(a[4], t_i32, "cu_q", 0, &cu) || read_dense(a[5], t_i32, "seq_lens", 0, &seq) ||
        read_tensor(a[8], t_bf16, "out", 0, &out) || read_dense(a[9], t_f32, "lse", 1, &lse) ||
        read_dense(a[10], t_u8, "workspace", 0, &ws) || heads(&q, "q", &ld_q) || heads(&out, "out", &ld_o) ||
        cache(&kc, &vc, &page_stride))
        return NULL;
    const int64_t T = q.size[0], H = q.size[1], D = q.size[2], reqs = seq.count;
    if (kc.size[3] != D || cu.count != reqs + 1 || table.dims != 2 || table.size[0] != reqs) {
        fail("q, the cache, block_table, cu_q and seq_lens do not fit one another");
        return NULL;
    }
    if (out.size[0] != T || out.size[1] != H || out.size[2] != D) {
        fail("out must have q's shape");
        return NULL;
    }
    if (a[9] != Py_None && (lse.dims != 2 || lse.size[0] != T || lse.size[1] != H)) {
        fail("lse must be [T, Hq]");
        return NULL;
    }
    if (rows(&table, reqs, table.size[1], "block_table", &ld_t))
        return NULL;
    const float scale = a[6] == Py_None ? 1.0f / sqrtf((float)D) : as_float(a[6]);
    const int64_t window = as_int(a[7]);
    const q2k_stream_t stream = as_stream(a[11]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_attn(q.p, ld_q, T, H, kc.size[1], D, kc.p, vc.p, kc.size[0], kc.size[2], page_stride, table.p,
                         table.size[1], ld_t, cu.p, seq.p, reqs, scale, window, out.p, ld_o, lse.p, ws.p, (size_t)ws.count,
                         stream));
}

/* T, Hq, Hkv, D */
static PyObject* py_attn_bytes(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    if (want_args(n, 4))
        return NULL;
    const int64_t T = as_int(a[0]), Hq = as_int(a[1]), Hkv = as_int(a[2]), D = as_int(a[3]);
    if (PyErr_Occurred())
        return NULL;
    return PyLong_FromSize_t(f_attn_bytes(T, Hq, Hkv, D));
}

/* residual, pre_w, eps, y, post_w, gate, alpha, residual_out, out, out_q8, stream */
static PyObject* py_norm(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor res, pre, y, post, gate, ro, out, q8;
    if (want_args(n, 11) || read_tensor(a[0], NULL, "residual", 0, &res))
        return NULL;
    const int s_type = type_of(&res, "residual");
    if (s_type < 0)
        return NULL;
    if (res.dims != 2) {
        fail("residual must be [T, dim] with dense rows");
        return NULL;
    }
    const int64_t T = res.size[0], dim = res.size[1];
    int64_t ld_res, ld_y = 0, ld_gate = 0, ld_ro, ld_out;
    int y_type = Q2K_F32;
    if (rows(&res, T, dim, "residual", &ld_res) || read_dense(a[1], t_f32, "pre_w", 0, &pre) ||
        read_tensor(a[3], NULL, "y", 1, &y) || read_dense(a[4], t_f32, "post_w", 1, &post))
        return NULL;
    if (a[3] != Py_None && ((y_type = type_of(&y, "y")) < 0 || rows(&y, T, dim, "y", &ld_y)))
        return NULL;
    if (read_tensor(a[5], a[3] == Py_None ? res.dtype : y.dtype, "gate", 1, &gate) ||
        read_tensor(a[7], res.dtype, "residual_out", 0, &ro) || rows(&ro, T, dim, "residual_out", &ld_ro) ||
        read_tensor(a[8], t_bf16, "out", 0, &out) || rows(&out, T, dim, "out", &ld_out) ||
        read_dense(a[9], t_u8, "out_q8", 1, &q8))
        return NULL;
    if (pre.count != dim || (a[4] != Py_None && post.count != dim)) {
        fail("a weight must have dim values");
        return NULL;
    }
    if (a[5] != Py_None) {
        const int last = gate.dims - 1;
        if (last < 0 || last > 1 || gate.size[last] != dim || (dim > 1 && gate.stride[last] != 1) ||
            (last == 1 && gate.size[0] != 1 && gate.size[0] != T)) {
            fail("gate must be [dim] or [T, dim] with dense rows");
            return NULL;
        }
        if (last == 1 && gate.size[0] > 1)
            ld_gate = gate.stride[0];
    }
    if (a[9] != Py_None && q8.count != T * (dim / 32) * 36) {
        fail("out_q8 must hold T q8_1 rows");
        return NULL;
    }
    const float eps = as_float(a[2]), alpha = as_float(a[6]);
    const q2k_stream_t stream = as_stream(a[10]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_norm(y.p, y_type, ld_y, post.p, gate.p, ld_gate, res.p, s_type, ld_res, alpha, pre.p, eps, T, dim, ro.p,
                         ld_ro, out.p, ld_out, q8.p, stream));
}

/* logits, topk, bias, score, n_group, topk_group, renorm, scale, ids, weights, expert_ptrs, ptrs, stream */
static PyObject* py_route(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor x, bias, ids, w, table, ptrs;
    int64_t ld;
    if (want_args(n, 13) || read_tensor(a[0], NULL, "logits", 0, &x))
        return NULL;
    const int type = type_of(&x, "logits");
    if (type < 0)
        return NULL;
    if (x.dims != 2) {
        fail("logits must be [m, E] with dense rows");
        return NULL;
    }
    const int64_t m = x.size[0], E = x.size[1], k = as_int(a[1]);
    if (PyErr_Occurred() || rows(&x, m, E, "logits", &ld) || read_dense(a[2], t_f32, "bias", 1, &bias) ||
        read_dense(a[8], t_i32, "ids", 0, &ids) || read_dense(a[9], t_f32, "weights", 0, &w) ||
        read_dense(a[10], t_i64, "expert_ptrs", 1, &table) || read_dense(a[11], t_i64, "ptrs", 1, &ptrs))
        return NULL;
    if ((a[2] != Py_None && bias.count != E) || (a[10] != Py_None && table.count != 3 * E)) {
        fail("bias must be [E], expert_ptrs [3, E]");
        return NULL;
    }
    if (ids.count != m * k || w.count != m * k || (a[11] != Py_None && ptrs.count != 3 * m * k)) {
        fail("ids, weights and ptrs must hold topk (3 * topk) entries per token");
        return NULL;
    }
    const int64_t groups = as_int(a[4]), kept = as_int(a[5]);
    const int score = (int)as_int(a[3]), renorm = PyObject_IsTrue(a[6]);
    const float scale = as_float(a[7]);
    const q2k_stream_t stream = as_stream(a[12]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_route(x.p, type, m, E, ld, bias.p, score, groups, kept, k, renorm, scale, ids.p, w.p, table.p, ptrs.p,
                          stream));
}

static int64_t blocks(int64_t n) { return (n + 127) / 128; }

/* x, block_rows, values, scales, stream; with swiglu, x holds gate and up and block_rows is 1 */
static PyObject* encode(PyObject* const* a, Py_ssize_t n, int swiglu)
{
    begin_call();
    Tensor x, q, scales;
    int64_t ldx, ldq, lds;
    const char* const name = swiglu ? "gate_up" : "x";
    if (want_args(n, 5) || read_tensor(a[0], NULL, name, 0, &x))
        return NULL;
    const int type = type_of(&x, name);
    if (type < 0)
        return NULL;
    const int64_t block_rows = as_int(a[1]);
    if (PyErr_Occurred())
        return NULL;
    if (x.dims != 2 || (swiglu && x.size[1] % 2)) {
        fail(swiglu ? "gate_up must be [rows, 2 N] with dense rows" : "x must be [rows, K] with dense rows");
        return NULL;
    }
    const int64_t T = x.size[0], K = swiglu ? x.size[1] / 2 : x.size[1];
    const int64_t s_rows = block_rows == 128 ? blocks(T) : T;
    if (rows(&x, T, x.size[1], name, &ldx) || read_tensor(a[2], t_e4m3, "values", 0, &q) ||
        rows(&q, T, K, "values", &ldq) || read_tensor(a[3], t_f32, "scales", 0, &scales) ||
        rows(&scales, s_rows, blocks(K), "scales", &lds))
        return NULL;
    const q2k_stream_t stream = as_stream(a[4]);
    if (PyErr_Occurred())
        return NULL;
    return status(swiglu ? f_swiglu(x.p, type, T, K, ldx, q.p, ldq, scales.p, lds, stream)
                         : f_quantize(x.p, type, T, K, ldx, block_rows, q.p, ldq, scales.p, lds, stream));
}

static PyObject* py_quantize(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    return encode(a, n, 0);
}

static PyObject* py_swiglu(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    return encode(a, n, 1);
}

/* x, x_scales, w, w_scales, out, stream */
static PyObject* py_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor x, xs, w, ws, out;
    int64_t ldx, ld_xs, ldy;
    if (want_args(n, 6) || read_tensor(a[0], t_e4m3, "x", 0, &x) || read_tensor(a[1], t_f32, "x_scales", 0, &xs) ||
        read_dense(a[2], t_e4m3, "w", 0, &w) || read_dense(a[3], t_f32, "w_scales", 0, &ws) ||
        read_tensor(a[4], NULL, "out", 0, &out))
        return NULL;
    const int type = type_of(&out, "out");
    if (type < 0)
        return NULL;
    if (x.dims != 2 || w.dims != 2 || w.size[1] != x.size[1]) {
        fail("x must be [m, K] and w [N, K]");
        return NULL;
    }
    const int64_t m = x.size[0], K = x.size[1], N = w.size[0];
    if (rows(&x, m, K, "x", &ldx) || rows(&xs, m, blocks(K), "x_scales", &ld_xs) || rows(&out, m, N, "out", &ldy))
        return NULL;
    if (ws.dims != 2 || ws.size[0] != blocks(N) || ws.size[1] != blocks(K)) {
        fail("w_scales must be [ceil(N / 128), ceil(K / 128)]");
        return NULL;
    }
    const q2k_stream_t stream = as_stream(a[5]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_gemm(x.p, m, K, ldx, xs.p, ld_xs, w.p, N, ws.p, out.p, type, ldy, stream));
}

/* x, ids, route_w, gate_up, gate_up_scales, down, down_scales, out, workspace, stream */
static PyObject* py_moe(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    begin_call();
    Tensor x, ids, w, gu, gs, down, ds, out, ws;
    int64_t ldx, ldy;
    if (want_args(n, 10) || read_tensor(a[0], t_bf16, "x", 0, &x) || read_dense(a[1], t_i32, "ids", 0, &ids) ||
        read_dense(a[2], t_f32, "route_w", 0, &w) || read_dense(a[3], t_e4m3, "gate_up", 0, &gu) ||
        read_dense(a[4], t_f32, "gate_up_scales", 0, &gs) || read_dense(a[5], t_e4m3, "down", 0, &down) ||
        read_dense(a[6], t_f32, "down_scales", 0, &ds) || read_tensor(a[7], NULL, "out", 0, &out) ||
        read_dense(a[8], t_u8, "workspace", 0, &ws))
        return NULL;
    const int type = type_of(&out, "out");
    if (type < 0)
        return NULL;
    if (x.dims != 2 || ids.dims != 2 || w.dims != 2 || ids.size[0] != x.size[0] || w.size[0] != x.size[0] ||
        w.size[1] != ids.size[1]) {
        fail("x must be [m, dim], ids and route_w [m, topk]");
        return NULL;
    }
    const int64_t m = x.size[0], dim = x.size[1], topk = ids.size[1];
    if (down.dims != 3 || down.size[1] != dim || gu.dims != 4 || gu.size[0] != down.size[0] || gu.size[1] != 2 ||
        gu.size[2] != down.size[2] || gu.size[3] != dim) {
        fail("gate_up must be [E, 2, inter, dim] and down [E, dim, inter]");
        return NULL;
    }
    const int64_t E = down.size[0], inter = down.size[2];
    if (gs.dims != 4 || gs.size[0] != E || gs.size[1] != 2 || gs.size[2] != blocks(inter) || gs.size[3] != blocks(dim) ||
        ds.dims != 3 || ds.size[0] != E || ds.size[1] != blocks(dim) || ds.size[2] != blocks(inter)) {
        fail("gate_up_scales must be [E, 2, ceil(inter / 128), ceil(dim / 128)] and down_scales "
             "[E, ceil(dim / 128), ceil(inter / 128)]");
        return NULL;
    }
    if (rows(&x, m, dim, "x", &ldx) || rows(&out, m, dim, "out", &ldy))
        return NULL;
    const q2k_stream_t stream = as_stream(a[9]);
    if (PyErr_Occurred())
        return NULL;
    return status(f_moe(x.p, m, dim, ldx, ids.p, w.p, topk, E, gu.p, gs.p, down.p, ds.p, inter, out.p, type, ldy, ws.p,
                        (size_t)ws.count, stream));
}

/* m, topk, dim, inter */
static PyObject* py_moe_bytes(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    if (want_args(n, 4))
        return NULL;
    const int64_t m = as_int(a[0]), topk = as_int(a[1]), dim = as_int(a[2]), inter = as_int(a[3]);
    if (PyErr_Occurred())
        return NULL;
    return PyLong_FromSize_t(f_moe_bytes(m, topk, dim, inter));
}

/* setup_fp8(e4m3, addresses of the five functions) */
static PyObject* py_setup_fp8(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    if (want_args(n, 2))
        return NULL;
    void* f[5];
    for (int i = 0; i < 5; ++i) {
        if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 5 ||
            !(f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[1], i)))) {
            if (!PyErr_Occurred())
                fail("five function addresses");
            return NULL;
        }
    }
    t_e4m3 = Py_NewRef(a[0]);
    *(void**)&f_quantize = f[0];
    *(void**)&f_swiglu = f[1];
    *(void**)&f_gemm = f[2];
    *(void**)&f_moe = f[3];
    *(void**)&f_moe_bytes = f[4];
    Py_RETURN_NONE;
}

/* setup((fp32, bf16, int32, int64, uint8), (addresses of the six functions), callable: the current device's index) */
static PyObject* py_setup(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    (void)self;
    if (want_args(n, 3))
        return NULL;
    void* f[6];
    if (!PyArg_ParseTuple(a[0], "OOOOO", &t_f32, &t_bf16, &t_i32, &t_i64, &t_u8))
        return NULL;
    for (int i = 0; i < 6; ++i) {
        if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 6 ||
            !(f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[1], i)))) {
            if (!PyErr_Occurred())
                fail("six function addresses");
            return NULL;
        }
    }
    Py_XSETREF(current_device, Py_NewRef(a[2]));
    Py_INCREF(t_f32);
    Py_INCREF(t_bf16);
    Py_INCREF(t_i32);
    Py_INCREF(t_i64);
    Py_INCREF(t_u8);
    *(void**)&f_plan = f[0];
    *(void**)&f_rope = f[1];
    *(void**)&f_attn = f[2];
    *(void**)&f_norm = f[3];
    *(void**)&f_route = f[4];
    *(void**)&f_attn_bytes = f[5];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, NULL},
    {"kv_page_plan", (PyCFunction)(void (*)(void))py_plan, METH_FASTCALL, NULL},
    {"kv_rope_store", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"kv_attention_bf16", (PyCFunction)(void (*)(void))py_attn, METH_FASTCALL, NULL},
    {"kv_attention_workspace_bytes", (PyCFunction)(void (*)(void))py_attn_bytes, METH_FASTCALL, NULL},
    {"norm_gate_residual", (PyCFunction)(void (*)(void))py_norm, METH_FASTCALL, NULL},
    {"moe_route_topk", (PyCFunction)(void (*)(void))py_route, METH_FASTCALL, NULL},
    {"setup_fp8", (PyCFunction)(void (*)(void))py_setup_fp8, METH_FASTCALL, NULL},
    {"fp8_quantize", (PyCFunction)(void (*)(void))py_quantize, METH_FASTCALL, NULL},
    {"swiglu_fp8_rows", (PyCFunction)(void (*)(void))py_swiglu, METH_FASTCALL, NULL},
    {"fp8_gemm", (PyCFunction)(void (*)(void))py_gemm, METH_FASTCALL, NULL},
    {"fp8_moe", (PyCFunction)(void (*)(void))py_moe, METH_FASTCALL, NULL},
    {"fp8_moe_workspace_bytes", (PyCFunction)(void (*)(void))py_moe_bytes, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_q2kcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__q2kcall(void)
{
    n_get_device = PyUnicode_InternFromString("get_device");
    n_dtype = PyUnicode_InternFromString("dtype");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    n_shape = PyUnicode_InternFromString("shape");
    n_stride = PyUnicode_InternFromString("stride");
    if (!n_get_device || !n_dtype || !n_data_ptr || !n_shape || !n_stride)
        return NULL;
    return PyModule_Create(&module);
}
