// Argument marshalling of the paged-cache calls in C++: a decode step makes them
// once per layer around kernels of a few microseconds, and the same checks in
// Python take longer than the kernels. Each function returns the library's
// status, or None when an argument is not plainly right (another device, type,
// shape or layout); the caller then takes the Python path, which names the error
// or accepts what this one does not.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "../../include/bitlinear.h"

namespace {

decltype(&bitlinear_rope_append) g_rope_append;
decltype(&bitlinear_paged_attention) g_paged_attention;

// The tensors of one call, read until one is not plainly right.
struct Reader {
    int device;
    bool ok = true;

    const at::Tensor *tensor(PyObject *o, at::ScalarType type)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        ok = t.is_cuda() && t.get_device() == device && t.scalar_type() == type;
        return &t;
    }

    // a contiguous tensor of the given sizes (-1: any)
    template <size_t N>
    const at::Tensor *dense(PyObject *o, at::ScalarType type, const int64_t (&sizes)[N])
    {
        const at::Tensor *t = tensor(o, type);
        if (ok)
            ok = t->dim() == static_cast<int64_t>(N) && t->is_contiguous();
        for (size_t i = 0; ok && i < N; ++i)
            ok = sizes[i] < 0 || t->size(i) == sizes[i];
        return t;
    }

    void *optional(PyObject *o, at::ScalarType type, int64_t n)
    {
        if (o == Py_None)
            return nullptr;
        const at::Tensor *t = dense(o, type, {n});
        return ok ? t->data_ptr() : nullptr;
    }

    struct Rows {
        void *p = nullptr;
        int64_t stride = 0, rows = 0, heads = 0;
    };

    // bf16 rows of whole heads, [T][heads * D] or [T][heads][D], each contiguous
    Rows rows(PyObject *o, int64_t D, int64_t T, int64_t heads)
    {
        Rows r;
        const at::Tensor *t = tensor(o, at::kBFloat16);
        if (!ok)
            return r;
        const int64_t n = t->dim();
        if (n == 3) {
            r.heads = t->size(1);
            ok = t->size(2) == D && t->stride(2) == 1 && (t->stride(1) == D || r.heads == 1);
        } else {
            ok = n == 2 && t->size(1) % D == 0 && t->stride(1) == 1;
            r.heads = ok ? t->size(1) / D : 0;
        }
        if (!ok)
            return r;
        r.rows = t->size(0);
        r.stride = r.rows > 1 ? t->stride(0) : r.heads * D;
        r.p = t->data_ptr();
        ok = r.heads > 0 && r.rows > 0 && (T < 0 || r.rows == T) && (heads < 0 || r.heads == heads);
        return r;
    }
};

struct Paged {
    bitlinear_kv_cache cache;
    bitlinear_seqs seqs;
};

// k_cache, v_cache, q_start, kv_len, page_table
Paged paged(Reader &in, PyObject *const *a)
{
    Paged p{};
    const at::Tensor *k = in.dense(a[0], at::kBFloat16, {-1, -1, -1, -1});
    if (!in.ok)
        return p;
    p.cache.pages = k->size(0);
    p.cache.kv_heads = k->size(1);
    p.cache.page = k->size(2);
    p.cache.head_dim = k->size(3);
    in.ok = p.cache.head_dim == 64 || p.cache.head_dim == 128;
    const at::Tensor *v = in.dense(
        a[1], at::kBFloat16, {p.cache.pages, p.cache.kv_heads, p.cache.page, p.cache.head_dim});
    const at::Tensor *table = in.dense(a[4], at::kInt, {-1, -1});
    if (!in.ok)
        return p;
    p.seqs.seqs = table->size(0);
    p.seqs.table_cols = table->size(1);
    const at::Tensor *start = in.dense(a[2], at::kInt, {p.seqs.seqs + 1});
    const at::Tensor *len = in.dense(a[3], at::kInt, {p.seqs.seqs});
    if (!in.ok)
        return p;
    p.cache.k_dev = k->data_ptr();
    p.cache.v_dev = v->data_ptr();
    p.seqs.q_start_dev = static_cast<const int32_t *>(start->data_ptr());
    p.seqs.kv_len_dev = static_cast<const int32_t *>(len->data_ptr());
    p.seqs.page_table_dev = static_cast<const int32_t *>(table->data_ptr());
    return p;
}

// A raw stream, or the current one for None.
void *stream_of(PyObject *o, int device)
{
    return o == Py_None ? c10::cuda::getCurrentCUDAStream(device).stream() : PyLong_AsVoidPtr(o);
}

// The status of a library call, which runs without the interpreter's lock: a launch
// waits while the stream's queue is full, and what empties the queue may need a Python
// thread (a host callback). The caller holds the tensors.
template <typename F>
PyObject *status(F call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// q, k, v, k_cache, v_cache, q_start, kv_len, page_table, inv_freq, q_out,
// q_gain, k_gain, eps, interleaved, stream
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 15 || g_rope_append == nullptr)
        Py_RETURN_NONE;
    try {
        Reader in{c10::cuda::current_device()};
        const Paged p = paged(in, a + 3);
        if (!in.ok)
            Py_RETURN_NONE;
        const int64_t D = p.cache.head_dim;
        const Reader::Rows q = in.rows(a[0], D, -1, -1);
        const Reader::Rows k = in.rows(a[1], D, q.rows, p.cache.kv_heads);
        const Reader::Rows v = in.rows(a[2], D, q.rows, p.cache.kv_heads);
        const Reader::Rows out = in.rows(a[9], D, q.rows, q.heads);
        const at::Tensor *f = in.dense(a[8], at::kFloat, {D / 2});
        const void *qg = in.optional(a[10], at::kFloat, D);
        const void *kg = in.optional(a[11], at::kFloat, D);
        const double eps = PyFloat_AsDouble(a[12]);
        const int interleaved = PyObject_IsTrue(a[13]);
        void *const stream = stream_of(a[14], in.device);
        if (!in.ok || PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        const auto *freq = static_cast<const float *>(f->data_ptr());
        return status([&] {
            return g_rope_append(q.p, q.stride, k.p, k.stride, v.p, v.stride, q.rows, q.heads,
                                 &p.cache, &p.seqs, freq, interleaved,
                                 static_cast<const float *>(qg), static_cast<const float *>(kg),
                                 static_cast<float>(eps), out.p, out.stride, stream);
        });
    } catch (const std::exception &) {
        Py_RETURN_NONE;
    }
}

// q, k_cache, v_cache, q_start, kv_len, page_table, scale (None: D ** -0.5),
// window, max_q_len (None: 0), y, lse, workspace, stream
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 13 || g_paged_attention == nullptr)
        Py_RETURN_NONE;
    try {
        Reader in{c10::cuda::current_device()};
        const Paged p = paged(in, a + 1);
        if (!in.ok)
            Py_RETURN_NONE;
        const int64_t D = p.cache.head_dim;
        const Reader::Rows q = in.rows(a[0], D, -1, -1);
        const Reader::Rows y = in.rows(a[9], D, q.rows, q.heads);
        const at::Tensor *lse =
            a[10] == Py_None ? nullptr : in.dense(a[10], at::kFloat, {q.rows, q.heads});
        const at::Tensor *ws = in.dense(a[11], at::kByte, {-1});
        const double scale =
            a[6] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : PyFloat_AsDouble(a[6]);
        const int64_t window = PyLong_AsLongLong(a[7]);
        const int64_t max_q = a[8] == Py_None ? 0 : PyLong_AsLongLong(a[8]);
        void *const stream = stream_of(a[12], in.device);
        if (!in.ok || PyErr_Occurred()) {
            PyErr_Clear();
            Py_RETURN_NONE;
        }
        float *const lse_p = lse == nullptr ? nullptr : static_cast<float *>(lse->data_ptr());
        void *const ws_p = ws->data_ptr();
        const size_t ws_bytes = static_cast<size_t>(ws->numel());
        return status([&] {
            return g_paged_attention(q.p, q.stride, q.rows, q.heads, &p.cache, &p.seqs,
                                     static_cast<float>(scale), window, max_q, y.p, y.stride, lse_p,
                                     ws_p, ws_bytes, stream);
        });
    } catch (const std::exception &) {
        Py_RETURN_NONE;
    }
}

// The addresses of the library's two functions.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "two addresses");
        return nullptr;
    }
    g_rope_append = reinterpret_cast<decltype(g_rope_append)>(PyLong_AsVoidPtr(a[0]));
    g_paged_attention = reinterpret_cast<decltype(g_paged_attention)>(PyLong_AsVoidPtr(a[1]));
    if (PyErr_Occurred())
        return nullptr;
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction method(F *f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {
    {"bind", method(bind), METH_FASTCALL, nullptr},
    {"rope_append", method(rope_append), METH_FASTCALL, nullptr},
    {"paged_attention", method(paged_attention), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&g_module); }
