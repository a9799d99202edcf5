// Argument marshalling of the paged-cache calls, for binding.py.
//
// Between kernels of a few microseconds the interpreter's share of a call
// counts: looking at six tensors' types, shapes, strides and addresses in
// Python and handing twenty arguments to ctypes takes about five microseconds
// on a Grace core, here half of one.  Each function checks what it reads and
// calls the C entry point; it returns the status, or None where an argument is
// not of the form that it handles -- binding.py then takes its own way, which
// names what is wrong or fills in what was left out.  No arithmetic, no
// allocation, no state but the entry points.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "w4a16.h"

namespace {

decltype(&w4a16_paged_map) g_map;
decltype(&w4a16_rope_append) g_append;
decltype(&w4a16_paged_attention) g_attention;
PyObject* g_current_stream;  // device index -> raw stream

const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// on the GPU `device`
bool on(const at::Tensor* t, int64_t device) { return t->is_cuda() && t->get_device() == device; }

// int32 vector of n entries
bool vector_of(PyObject* o, int64_t n, int64_t device, int32_t** p) {
    const at::Tensor* t = tensor_of(o);
    if (!t || t->scalar_type() != at::kInt || !on(t, device) || t->dim() != 1 || t->size(0) != n ||
        (n > 1 && t->stride(0) != 1))
        return false;
    *p = static_cast<int32_t*>(t->data_ptr());
    return true;
}

struct Table {
    int32_t* p;
    int64_t rows, columns, stride;
};
bool table_of(PyObject* o, int64_t device, Table* x) {
    const at::Tensor* t = tensor_of(o);
    if (!t || t->scalar_type() != at::kInt || !on(t, device) || t->dim() != 2) return false;
    x->rows = t->size(0), x->columns = t->size(1), x->stride = t->stride(0);
    if (x->columns > 1 && t->stride(1) != 1) return false;
    if (x->rows <= 1 && x->stride < x->columns) x->stride = x->columns;
    x->p = static_cast<int32_t*>(t->data_ptr());
    return true;
}

// bf16 [rows, heads, dim], dim contiguous
struct Rows {
    uint16_t* p = nullptr;
    int64_t n = 0, heads = 0, dim = 0, row = 0, head = 0;
    int64_t device = -1;
};
bool rows_of(PyObject* o, Rows* x) {
    const at::Tensor* t = tensor_of(o);
    if (!t || t->scalar_type() != at::kBFloat16 || !t->is_cuda() || t->dim() != 3 || t->stride(2) != 1) return false;
    x->n = t->size(0), x->heads = t->size(1), x->dim = t->size(2);
    x->row = t->stride(0), x->head = t->stride(1);
    x->device = t->get_device();
    x->p = static_cast<uint16_t*>(t->data_ptr());
    return true;
}

// the raw stream given, or the current one of `device`
bool stream_of(PyObject* o, int64_t device, void** s) {
    if (o != Py_None) {
        *s = PyLong_AsVoidPtr(o);
        return !PyErr_Occurred();
    }
    PyObject* index = PyLong_FromLongLong(device);
    PyObject* raw = index ? PyObject_CallOneArg(g_current_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!raw) return false;
    *s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    return !PyErr_Occurred();
}

bool integer(PyObject* o, int64_t* v) {
    if (!PyLong_Check(o)) return false;
    *v = PyLong_AsLongLong(o);
    return !PyErr_Occurred();
}

// a list or tuple of at most four whole numbers; None: one axis, no array
struct Sections {
    int32_t n[4];
    const int32_t* p = nullptr;
    int axes = 1;
};
bool sections_of(PyObject* o, Sections* x) {
    if (o == Py_None) return true;
    if (!PyList_CheckExact(o) && !PyTuple_CheckExact(o)) return false;
    const Py_ssize_t size = PySequence_Fast_GET_SIZE(o);
    if (size < 1 || size > 4) return false;
    for (Py_ssize_t i = 0; i < size; ++i) {
        int64_t v;
        if (!integer(PySequence_Fast_GET_ITEM(o, i), &v) || v < INT32_MIN || v > INT32_MAX) return false;
        x->n[i] = static_cast<int32_t>(v);
    }
    x->p = x->n;
    x->axes = static_cast<int>(size);
    return true;
}

PyObject* other_form() {  // not for here: no error is left behind
    PyErr_Clear();
    Py_RETURN_NONE;
}

template <class Call>
PyObject* status_of(Call call) {
    w4a16_status rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// (ctx_len, new_len, block_table, free_blocks, free_head, page, num_blocks, tokens, out, stream)
PyObject* paged_map(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 10 || !g_map) return other_form();
    try {
        const at::Tensor* first = tensor_of(a[0]);
        if (!first || first->dim() != 1 || !PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 5) return other_form();
        const int64_t B = first->size(0), dev = first->get_device();
        const at::Tensor* free_t = tensor_of(a[3]);
        if (!free_t || free_t->dim() != 1) return other_form();
        const int64_t F = free_t->size(0);
        int32_t *ctx, *fresh, *free_blocks, *head, *slots, *positions, *row_start, *kv_len, *head_out;
        Table t;
        int64_t page, blocks, tokens;
        void* stream;
        if (!integer(a[5], &page) || !integer(a[6], &blocks) || !integer(a[7], &tokens) || !vector_of(a[0], B, dev, &ctx) ||
            !vector_of(a[1], B, dev, &fresh) || !table_of(a[2], dev, &t) || t.rows != B || !vector_of(a[3], F, dev, &free_blocks) ||
            !vector_of(a[4], 1, dev, &head) || !vector_of(PyTuple_GET_ITEM(a[8], 0), tokens, dev, &slots) ||
            !vector_of(PyTuple_GET_ITEM(a[8], 1), tokens, dev, &positions) ||
            !vector_of(PyTuple_GET_ITEM(a[8], 2), B + 1, dev, &row_start) ||
            !vector_of(PyTuple_GET_ITEM(a[8], 3), B, dev, &kv_len) ||
            !vector_of(PyTuple_GET_ITEM(a[8], 4), 1, dev, &head_out) || B > INT32_MAX || t.columns > INT32_MAX ||
            page > INT32_MAX || page < INT32_MIN || !stream_of(a[9], dev, &stream))
            return other_form();
        return status_of([&] {
            return g_map(ctx, fresh, static_cast<int>(B), t.p, t.stride, static_cast<int>(t.columns), free_blocks, F, head,
                         static_cast<int>(page), blocks, slots, positions, tokens, row_start, kv_len, head_out, stream);
        });
    } catch (...) {
        return other_form();
    }
}

// (q, k, v, positions, inv_freq, slots, cache address, cache heads, cache device, sections, flags, q_out, stream)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13 || !g_append) return other_form();
    try {
        Rows q, out, k, v;
        int32_t *slots = nullptr, *positions;
        int64_t cache = 0, heads = 0, cache_device, flags;
        Sections sections;
        if (a[0] != Py_None) {
            if (!rows_of(a[0], &q) || !rows_of(a[11], &out) || out.n != q.n || out.heads != q.heads || out.dim != q.dim ||
                out.device != q.device)
                return other_form();
        }
        if (a[6] != Py_None) {
            if (!integer(a[6], &cache) || !integer(a[7], &heads) || !integer(a[8], &cache_device) || !rows_of(a[1], &k) || !rows_of(a[2], &v) ||
                k.heads != heads || v.heads != heads || v.n != k.n || v.dim != k.dim || k.device != cache_device ||
                v.device != cache_device || (q.p && (q.n != k.n || q.dim != k.dim || q.device != cache_device)) ||
                !vector_of(a[5], k.n, cache_device, &slots))
                return other_form();
        }
        const Rows& any = q.p ? q : k;
        const at::Tensor* pos = tensor_of(a[3]);
        const at::Tensor* freq = tensor_of(a[4]);
        void* stream;
        if (!any.p || !pos || !freq || !sections_of(a[9], &sections) || !integer(a[10], &flags) ||
            freq->scalar_type() != at::kFloat || !on(freq, any.device) || freq->dim() != 1 || !freq->is_contiguous())
            return other_form();
        if (pos->dim() == 1) {
            if (sections.axes != 1 || !vector_of(a[3], any.n, any.device, &positions)) return other_form();
        } else {
            if (pos->dim() != 2 || pos->scalar_type() != at::kInt || !on(pos, any.device) || !pos->is_contiguous() || pos->size(0) != sections.axes ||
                pos->size(1) != any.n)
                return other_form();
            positions = static_cast<int32_t*>(pos->data_ptr());
        }
        if (any.n == 0 || q.heads > INT32_MAX || freq->size(0) > INT32_MAX / 2 || !stream_of(a[12], any.device, &stream))
            return other_form();
        const int rotary = 2 * static_cast<int>(freq->size(0));
        const float* f = static_cast<const float*>(freq->data_ptr());
        return status_of([&] {
            return g_append(q.p, q.row, q.head, out.p, out.row, out.head, static_cast<int>(q.heads), k.p, k.row, k.head, v.p, v.row,
                            v.head, positions, any.n, f, sections.p, sections.axes, rotary,
                            static_cast<int>(any.dim), static_cast<unsigned>(flags), slots,
                            reinterpret_cast<const w4a16_kv_cache*>(cache), any.n, stream);
        });
    } catch (...) {
        return other_form();
    }
}

// (q, cache address, cache dim, cache device, block_table, kv_len, scale, window, out, lse, workspace, stream)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 12 || !g_attention) return other_form();
    try {
        Rows q, out;
        Table t;
        int32_t* lengths;
        int64_t cache, dim, device, window;
        if (!rows_of(a[0], &q) || !integer(a[1], &cache) || !integer(a[2], &dim) || q.dim != dim || !integer(a[3], &device) ||
            q.device != device || !table_of(a[4], device, &t) || t.rows != q.n || !vector_of(a[5], q.n, device, &lengths) ||
            !integer(a[7], &window) || !rows_of(a[8], &out) || out.n != q.n || out.heads != q.heads || out.dim != dim ||
            out.device != device)
            return other_form();
        const at::Tensor *lse = tensor_of(a[9]), *ws = tensor_of(a[10]);
        if (!lse || !ws || lse->scalar_type() != at::kFloat || !on(lse, device) || lse->dim() != 2 || lse->size(0) != q.n ||
            lse->size(1) != q.heads || !lse->is_contiguous() || !on(ws, device) || !ws->is_contiguous())
            return other_form();
        const double scale = PyFloat_AsDouble(a[6]);
        void* stream;
        if (PyErr_Occurred() || q.n > INT32_MAX || q.heads > INT32_MAX || t.columns > INT32_MAX || window > INT32_MAX ||
            window < INT32_MIN || !stream_of(a[11], device, &stream))
            return other_form();
        float* l = static_cast<float*>(lse->data_ptr());
        void* w = ws->data_ptr();
        const size_t bytes = ws->nbytes();
        return status_of([&] {
            return g_attention(q.p, q.row, q.head, reinterpret_cast<const w4a16_kv_cache*>(cache), t.p, t.stride,
                               static_cast<int>(t.columns), lengths, static_cast<int>(q.n), static_cast<int>(q.heads),
                               static_cast<float>(scale), static_cast<int>(window), out.p, out.row, out.head, l, w, bytes, stream);
        });
    } catch (...) {
        return other_form();
    }
}

// bind(map address, append address, attention address, current-stream function)
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long m, p, t;
    PyObject* f;
    if (!PyArg_ParseTuple(args, "KKKO", &m, &p, &t, &f)) return nullptr;
    g_map = reinterpret_cast<decltype(g_map)>(m);
    g_append = reinterpret_cast<decltype(g_append)>(p);
    g_attention = reinterpret_cast<decltype(g_attention)>(t);
    Py_INCREF(f);
    Py_XDECREF(g_current_stream);
    g_current_stream = f;
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"paged_map", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_map)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(paged_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&g_module); }
