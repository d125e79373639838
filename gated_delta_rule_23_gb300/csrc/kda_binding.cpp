// The decoder-step operators' short way from Python to libkda.so.
//
// A decode step's kernels take a few microseconds; reading a dozen tensors' types, shapes, strides and pointers through
// Python attributes takes longer than that.  These functions read them here and call the C ABI.  They only ever accept:
// whatever is not exactly what the call expects (a wrong type, shape, device or layout, another current device) makes
// them return None before anything is launched, and the caller goes through the full checks in step.py, which either
// make the call or say what is wrong.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <vector>

#include "kda.h"

namespace {

decltype(&kda_kv_append) g_append;
decltype(&kda_window_attn) g_attn;
decltype(&kda_window_attn_ws) g_attn_ws;
decltype(&kda_beam_select) g_beam;
decltype(&kda_beam_select_ws) g_beam_ws;
decltype(&kda_state_reorder) g_reorder;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The device of the call: that of its first tensor, which has to be the current one.  -1: none.
int device_of(const at::Tensor *t)
{
    if (!t || !t->is_cuda())
        return -1;
    const int dev = t->get_device();
    return dev == c10::cuda::current_device() ? dev : -1;
}

bool dense(const at::Tensor *t, at::ScalarType type, at::IntArrayRef shape, int dev)
{
    return t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == shape &&
           t->is_contiguous();
}

// A [B, T, heads, dim] bf16 tensor of evenly spaced tokens: its token stride, or -1.
int64_t rows(const at::Tensor *t, int64_t b, int64_t n, int dev)
{
    if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != at::kBFloat16 || t->dim() != 4 ||
        t->size(0) != b || t->size(1) != n || t->numel() == 0)
        return -1;
    const int64_t heads = t->size(2), dim = t->size(3);
    if (t->is_contiguous())
        return heads * dim;
    const int64_t step = n > 1 ? t->stride(1) : (b > 1 ? t->stride(0) : heads * dim);
    if ((dim > 1 && t->stride(3) != 1) || (heads > 1 && t->stride(2) != dim) || (b > 1 && t->stride(0) != n * step) ||
        step % 8 || step < heads * dim)
        return -1;
    return step;
}

bool stream_of(PyObject *o, int dev, kda_stream_t *s)
{
    if (o == Py_None) {
        *s = reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
        return true;
    }
    if (!PyLong_Check(o))
        return false;
    *s = static_cast<kda_stream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}

bool int_of(PyObject *o, int64_t lo, int64_t hi, int *v)
{
    if (!PyLong_Check(o))
        return false;
    int over = 0;
    const int64_t x = PyLong_AsLongLongAndOverflow(o, &over);
    if (over || x < lo || x > hi)
        return false;
    *v = (int)x;
    return true;
}

struct Cache {
    void *k, *v;
    const int32_t *table, *lens;
    const int64_t *cu;
    int N, hkv, dim, page, max_pages;
    int64_t pages;
};

bool cache_of(PyObject *ko, PyObject *vo, PyObject *to, PyObject *lo, PyObject *co, int64_t b, int dev, Cache *c)
{
    const at::Tensor *k = tensor(ko), *v = tensor(vo), *table = tensor(to), *lens = tensor(lo), *cu = tensor(co);
    if (!k || !table || k->dim() != 4 || table->dim() != 2 || k->size(1) > INT32_MAX || k->size(2) > INT32_MAX ||
        table->size(1) > INT32_MAX || !dense(k, at::kBFloat16, k->sizes(), dev) ||
        !dense(v, at::kBFloat16, k->sizes(), dev))
        return false;
    int64_t n = b;
    c->cu = nullptr;
    if (co != Py_None) {
        if (!cu || b != 1 || cu->dim() != 1 || cu->numel() < 2 || !dense(cu, at::kLong, cu->sizes(), dev))
            return false;
        n = cu->numel() - 1;
        c->cu = static_cast<const int64_t *>(cu->data_ptr());
    }
    if (n > INT32_MAX || !dense(table, at::kInt, {n, table->size(1)}, dev) || !dense(lens, at::kInt, {n}, dev))
        return false;
    c->k = k->data_ptr(), c->v = v->data_ptr();
    c->table = static_cast<const int32_t *>(table->data_ptr());
    c->lens = static_cast<const int32_t *>(lens->data_ptr());
    c->N = (int)n, c->hkv = (int)k->size(1), c->page = (int)k->size(2), c->dim = (int)k->size(3);
    c->pages = k->size(0), c->max_pages = (int)table->size(1);
    return true;
}

// Runs f, which gives a status or -1 for "not here".
template <typename F> PyObject *answer(F f)
{
    int rc = -1;
    try {
        rc = f();
    } catch (...) {
        rc = -1;
    }
    if (PyErr_Occurred())
        PyErr_Clear();
    if (rc < 0)
        Py_RETURN_NONE;
    return PyLong_FromLong(rc);
}

// k, v, k_cache, v_cache, block_table, kv_lens, cos, sin, interleaved, q, q_out, cu_seqlens, stream
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer([&]() -> int {
        if (n != 13)
            return -1;
        const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]);
        const int dev = device_of(k);
        if (dev < 0 || k->dim() != 4)
            return -1;
        const int64_t b = k->size(0), t = k->size(1), ks = rows(k, b, t, dev), vs = rows(v, b, t, dev);
        Cache c;
        if (ks < 0 || vs < 0 || v->sizes() != k->sizes() || !cache_of(a[2], a[3], a[4], a[5], a[11], b, dev, &c) ||
            k->size(2) != c.hkv || k->size(3) != c.dim)
            return -1;
        const float *cos = nullptr, *sin = nullptr;
        int64_t rotary = 0, positions = 0;
        if (a[6] != Py_None || a[7] != Py_None) {
            const at::Tensor *x = tensor(a[6]), *y = tensor(a[7]);
            if (!x || x->dim() != 2 || x->size(1) > 1024 || !dense(x, at::kFloat, x->sizes(), dev) ||
                !dense(y, at::kFloat, x->sizes(), dev))
                return -1;
            cos = static_cast<const float *>(x->data_ptr()), sin = static_cast<const float *>(y->data_ptr());
            positions = x->size(0), rotary = 2 * x->size(1);
        }
        const int inter = PyObject_IsTrue(a[8]);
        const void *q = nullptr;
        void *q_out = nullptr;
        int64_t hq = 0, qs = 0;
        if (a[9] != Py_None || a[10] != Py_None) {
            const at::Tensor *x = tensor(a[9]), *y = tensor(a[10]);
            qs = rows(x, b, t, dev);
            if (qs < 0 || x->size(3) != c.dim || x->size(2) > INT32_MAX || !dense(y, at::kBFloat16, x->sizes(), dev))
                return -1;
            q = x->data_ptr(), q_out = y->data_ptr(), hq = x->size(2);
        }
        kda_stream_t s;
        if (inter < 0 || !stream_of(a[12], dev, &s))
            return -1;
        return g_append(k->data_ptr(), ks, v->data_ptr(), vs, c.k, c.v, c.table, c.lens, cos, sin, (int)rotary, positions,
                        inter, q, qs, q_out, c.cu, c.N, t, (int)hq, c.hkv, c.dim, c.pages, c.page, c.max_pages, s);
    });
}

// q, k_cache, v_cache, block_table, kv_lens, out, window, sinks, scale, lse, cu_seqlens, stream, workspace
PyObject *window_attn(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer([&]() -> int {
        if (n != 13)
            return -1;
        const at::Tensor *q = tensor(a[0]);
        const int dev = device_of(q);
        if (dev < 0 || q->dim() != 4)
            return -1;
        const int64_t b = q->size(0), t = q->size(1), qs = rows(q, b, t, dev);
        Cache c;
        if (qs < 0 || q->size(2) > INT32_MAX || !cache_of(a[1], a[2], a[3], a[4], a[10], b, dev, &c) || q->size(3) != c.dim)
            return -1;
        const at::Tensor *out = tensor(a[5]), *lse = tensor(a[9]), *ws = tensor(a[12]);
        if (!dense(out, at::kBFloat16, q->sizes(), dev) ||
            (a[9] != Py_None && !dense(lse, at::kFloat, {b, t, q->size(2)}, dev)) ||
            (a[12] != Py_None && (!ws || !dense(ws, at::kByte, ws->sizes(), dev))))
            return -1;
        int window, sinks;
        kda_stream_t s;
        if (!int_of(a[6], 1, INT32_MAX, &window) || !int_of(a[7], 0, INT32_MAX, &sinks) || !stream_of(a[11], dev, &s))
            return -1;
        const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)c.dim) : PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred())
            return -1;
        float *lp = lse ? static_cast<float *>(lse->data_ptr()) : nullptr;
        if (ws)
            return g_attn_ws(q->data_ptr(), qs, c.k, c.v, c.table, c.lens, out->data_ptr(), lp, (float)scale, window, sinks,
                             c.cu, c.N, t, (int)q->size(2), c.hkv, c.dim, c.pages, c.page, c.max_pages, ws->data_ptr(),
                             (size_t)ws->numel(), s);
        return g_attn(q->data_ptr(), qs, c.k, c.v, c.table, c.lens, out->data_ptr(), lp, (float)scale, window, sinks, c.cu,
                      c.N, t, (int)q->size(2), c.hkv, c.dim, c.pages, c.page, c.max_pages, s);
    });
}

// logits, beam_scores, scores, tokens, parents, finished, eos, stream, workspace
PyObject *beam_select(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer([&]() -> int {
        if (n != 9)
            return -1;
        const at::Tensor *l = tensor(a[0]), *tokens = tensor(a[3]), *fin = tensor(a[5]), *ws = tensor(a[8]);
        const int dev = device_of(l);
        if (dev < 0 || l->dim() != 3 || !tokens || tokens->dim() != 2 || l->numel() == 0)
            return -1;
        const int64_t b = l->size(0), w = l->size(1), v = l->size(2), k = tokens->size(1);
        const bool half = l->scalar_type() == at::kBFloat16;
        if ((!half && l->scalar_type() != at::kFloat) || b > INT32_MAX || w > INT32_MAX || v > INT32_MAX || k > INT32_MAX)
            return -1;
        const int64_t step = w > 1 ? l->stride(1) : (b > 1 ? l->stride(0) : v);
        if ((v > 1 && l->stride(2) != 1) || (b > 1 && l->stride(0) != w * step) || step < v)
            return -1;
        const at::Tensor *bs = tensor(a[1]), *scores = tensor(a[2]), *parents = tensor(a[4]);
        if (!dense(bs, at::kFloat, {b, w}, dev) || !dense(scores, at::kFloat, {b, k}, dev) ||
            !dense(tokens, at::kInt, {b, k}, dev) || !dense(parents, at::kInt, {b, k}, dev))
            return -1;
        if (a[5] != Py_None && !dense(fin, at::kByte, {b, w}, dev) && !dense(fin, at::kBool, {b, w}, dev))
            return -1;
        if (a[8] != Py_None && (!ws || !dense(ws, at::kByte, ws->sizes(), dev)))
            return -1;
        int eos;
        kda_stream_t s;
        if (!int_of(a[6], INT32_MIN, INT32_MAX, &eos) || !stream_of(a[7], dev, &s))
            return -1;
        const uint8_t *fp = fin ? static_cast<const uint8_t *>(fin->data_ptr()) : nullptr;
        const kda_dtype_t dtype = half ? KDA_DTYPE_BF16 : KDA_DTYPE_FP32;
        float *sp = static_cast<float *>(scores->data_ptr());
        int32_t *tp = static_cast<int32_t *>(tokens->data_ptr()), *pp = static_cast<int32_t *>(parents->data_ptr());
        const float *bp = static_cast<const float *>(bs->data_ptr());
        if (ws)
            return g_beam_ws(l->data_ptr(), dtype, step, bp, fp, eos, sp, tp, pp, (int)b, (int)w, (int)v, (int)k,
                             ws->data_ptr(), (size_t)ws->numel(), s);
        return g_beam(l->data_ptr(), dtype, step, bp, fp, eos, sp, tp, pp, (int)b, (int)w, (int)v, (int)k, s);
    });
}

// src (list or tuple of tensors), dst (the same, or None: in place), parents, beams, stream
PyObject *state_reorder(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return answer([&]() -> int {
        if (n != 5 || !(PyList_Check(a[0]) || PyTuple_Check(a[0])) ||
            !(a[1] == Py_None || PyList_Check(a[1]) || PyTuple_Check(a[1])))
            return -1;
        const at::Tensor *parents = tensor(a[2]);
        const int dev = device_of(parents);
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
        if (dev < 0 || (a[1] != Py_None && PySequence_Fast_GET_SIZE(a[1]) != count) || count > 4096)
            return -1;
        const int64_t rows_n = parents->numel();
        if (rows_n < 1 || rows_n > INT32_MAX || !dense(parents, at::kInt, {rows_n}, dev))
            return -1;
        std::vector<const void *> src(count);
        std::vector<void *> dst(count);
        std::vector<int64_t> bytes(count);
        for (Py_ssize_t i = 0; i < count; i++) {
            const at::Tensor *x = tensor(PySequence_Fast_GET_ITEM(a[0], i));
            const at::Tensor *y = a[1] == Py_None ? x : tensor(PySequence_Fast_GET_ITEM(a[1], i));
            if (!x || x->dim() < 1 || x->size(0) != rows_n || !dense(x, x->scalar_type(), x->sizes(), dev) ||
                !dense(y, x->scalar_type(), x->sizes(), dev))
                return -1;
            src[i] = x->data_ptr(), dst[i] = y->data_ptr();
            bytes[i] = x->numel() / rows_n * (int64_t)x->element_size();
        }
        int beams;
        kda_stream_t s;
        if (!int_of(a[3], INT32_MIN, INT32_MAX, &beams) || !stream_of(a[4], dev, &s))
            return -1;
        return g_reorder(src.data(), dst.data(), bytes.data(), (int)count, static_cast<const int32_t *>(parents->data_ptr()),
                         (int)rows_n, beams, s);
    });
}

// Addresses of libkda.so's entry points, in the order of the globals above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    void *p[6];
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind takes 6 addresses");
        return nullptr;
    }
    for (int i = 0; i < 6; i++) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred())
            return nullptr;
    }
    g_append = reinterpret_cast<decltype(g_append)>(p[0]);
    g_attn = reinterpret_cast<decltype(g_attn)>(p[1]);
    g_attn_ws = reinterpret_cast<decltype(g_attn_ws)>(p[2]);
    g_beam = reinterpret_cast<decltype(g_beam)>(p[3]);
    g_beam_ws = reinterpret_cast<decltype(g_beam_ws)>(p[4]);
    g_reorder = reinterpret_cast<decltype(g_reorder)>(p[5]);
    Py_RETURN_NONE;
}

template <typename F> PyCFunction as_c(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)); }

PyMethodDef methods[] = {{"bind", as_c(bind), METH_FASTCALL, nullptr},
                         {"kv_append", as_c(kv_append), METH_FASTCALL, nullptr},
                         {"window_attn", as_c(window_attn), METH_FASTCALL, nullptr},
                         {"beam_select", as_c(beam_select), METH_FASTCALL, nullptr},
                         {"state_reorder", as_c(state_reorder), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "kda_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_binding() { return PyModule_Create(&module_def); }
