// fd_torch.cpp - what attention.py does for a call whose arguments are all in order, in C++: the
// tensors' addresses, sizes and strides read and checked, outputs allocated, the C ABI called. A
// decoding step's calls take 2 to 10 us on the GPU; in Python this costs 14 to 17 us a call.
//
// Each function returns its result; the status (an int, not 0) of a call that the library refused;
// or None where an argument is not plainly in order or is not handled here (a given stream, another
// current device, a subclass of Tensor), and attention.py then does the same in Python, where it
// also finds the words for what is wrong.
#include <Python.h>

#include <cmath>
#include <cstdint>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fd.h"

namespace {

// The entry points, as the ctypes binding has loaded them (init).
decltype(&fd_rope) g_rope;
decltype(&fd_rope_append) g_append;
decltype(&fd_paged_attention) g_attention;

const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// A call's tensors: of one device, the current one. `ok` turns false at the first that is not in order.
struct Call {
    bool ok = true;
    c10::DeviceIndex dev = -1;

    const at::Tensor *take(PyObject *o, at::ScalarType type, int64_t dims) {
        const at::Tensor *t = ok ? tensor(o) : nullptr;
        ok = t && t->is_cuda() && t->layout() == at::kStrided && t->scalar_type() == type && t->dim() == dims &&
             (dev < 0 || t->get_device() == dev);
        if (!ok) return nullptr;
        if (dev < 0) {
            dev = t->get_device();
            ok = dev == c10::cuda::current_device();
        }
        return ok ? t : nullptr;
    }
    // bf16 [tokens, heads, head_dim]; negative: any size.
    const at::Tensor *heads(PyObject *o, fd_heads *h, int64_t n, int64_t heads, int64_t d) {
        const at::Tensor *t = take(o, at::kBFloat16, 3);
        if (!t) return nullptr;
        const auto size = t->sizes(), stride = t->strides();
        ok = stride[2] == 1 && (n < 0 || size[0] == n) && (heads < 0 || size[1] == heads) && (d < 0 || size[2] == d) &&
             size[0] <= INT32_MAX && size[1] <= INT32_MAX && size[2] <= INT32_MAX;
        if (!ok) return nullptr;
        *h = {t->data_ptr(), size[0] > 1 ? stride[0] : 0, size[1] > 1 ? stride[1] : 0, (int)size[1]};
        return t;
    }
    void *flat(PyObject *o, at::ScalarType type, int64_t n, int64_t *size = nullptr) {
        const at::Tensor *t = take(o, type, 1);
        ok = t && (n < 0 || t->size(0) == n) && t->is_contiguous();
        if (!ok) return nullptr;
        if (size) *size = t->size(0);
        return t->data_ptr();
    }
    void cache(PyObject *ko, PyObject *vo, fd_paged_cache *c) {
        const at::Tensor *k = take(ko, at::kBFloat16, 4), *v = take(vo, at::kBFloat16, 4);
        ok = k && v && k->sizes() == v->sizes() && k->stride(3) == 1 && v->stride(3) == 1;
        if (!ok) return;
        const auto size = k->sizes(), a = k->strides(), b = v->strides();
        for (const int64_t n : size) ok = ok && n <= INT32_MAX;
        *c = {k->data_ptr(), v->data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], (int)size[0], (int)size[1], (int)size[2],
              (int)size[3]};
    }
    void batch(PyObject *qs, PyObject *kl, PyObject *bt, int64_t total_q, int64_t max_q, fd_paged_batch *b) {
        int64_t n = 0;
        const void *kv = flat(kl, at::kInt, -1, &n);
        const void *start = ok ? flat(qs, at::kInt, n + 1) : nullptr;
        const at::Tensor *t = take(bt, at::kInt, 2);
        if (!t) return;
        const auto size = t->sizes(), stride = t->strides();
        ok = size[0] == n && (stride[1] == 1 || size[1] <= 1) && stride[0] <= INT32_MAX && size[1] <= INT32_MAX &&
             n < INT32_MAX;
        if (!ok) return;
        *b = {static_cast<const int *>(start), static_cast<const int *>(kv), t->const_data_ptr<int>(),
              (int)(n > 1 ? stride[0] : size[1]), (int)n, (int)total_q, (int)max_q, (int)size[1]};
    }
    // An output of the size and device of `like`: given, or new.
    at::Tensor output(PyObject *o, const at::Tensor &like, fd_heads *h) {
        const auto size = like.sizes();
        if (o != Py_None) {
            const at::Tensor *t = heads(o, h, size[0], size[1], size[2]);
            return t ? *t : at::Tensor();
        }
        at::Tensor t = at::empty(size, like.options());
        *h = {t.data_ptr(), size[1] * size[2], size[2], (int)size[1]};
        return t;
    }
    fd_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

bool number(PyObject *o, double *x) {
    *x = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyLong_Check(o) ? PyLong_AsDouble(o) : (PyErr_SetNone(PyExc_TypeError), 0);
    if (!PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
bool whole(PyObject *o, int64_t *x) {
    *x = PyLong_Check(o) ? PyLong_AsLongLong(o) : (PyErr_SetNone(PyExc_TypeError), 0);
    if (!PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
// 0 or 1; -1: neither True nor False.
int truth(PyObject *o) { return o == Py_True ? 1 : o == Py_False ? 0 : -1; }

PyObject *wrap(PyObject *given, const at::Tensor &t) { return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(t); }

// rope(q, k | None, positions, inv_freq, interleaved, scale, q_out | None, k_out | None) -> (q_out, k_out)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    double scale = 0;
    const int interleaved = n_args == 8 ? truth(a[4]) : -1;
    if (interleaved < 0 || !number(a[5], &scale) || (a[1] == Py_None && a[7] != Py_None)) Py_RETURN_NONE;
    Call c;
    fd_heads qh{}, kh{}, qo{}, ko{};
    const at::Tensor *q = c.heads(a[0], &qh, -1, -1, -1);
    if (!q) Py_RETURN_NONE;
    const int64_t n = q->size(0), d = q->size(2);
    const void *pos = c.flat(a[2], at::kInt, n);
    int64_t pairs = 0;
    const void *freq = c.ok ? c.flat(a[3], at::kDouble, -1, &pairs) : nullptr;
    const bool with_k = a[1] != Py_None;
    const at::Tensor *k = with_k ? c.heads(a[1], &kh, n, -1, d) : nullptr;
    if (!c.ok || pairs < 1 || pairs > d / 2) Py_RETURN_NONE;
    at::Tensor k_out, q_out;
    if (with_k) k_out = c.output(a[7], *k, &ko);
    if (c.ok) q_out = c.output(a[6], *q, &qo);
    if (!c.ok) Py_RETURN_NONE;
    int st;
    const fd_stream_t stream = c.stream();
    Py_BEGIN_ALLOW_THREADS;
    st = g_rope(&qh, with_k ? &kh : nullptr, &qo, with_k ? &ko : nullptr, static_cast<const int *>(pos),
                static_cast<const double *>(freq), (int)n, (int)d, (int)(2 * pairs), interleaved, (float)scale, stream);
    Py_END_ALLOW_THREADS;
    if (st) return PyLong_FromLong(st);
    PyObject *first = wrap(a[6], q_out);
    if (!first) return nullptr;
    PyObject *second = with_k ? wrap(a[7], k_out) : Py_NewRef(Py_None);
    PyObject *both = second ? PyTuple_New(2) : nullptr;
    if (!both) {
        Py_DECREF(first);
        Py_XDECREF(second);
        return nullptr;
    }
    PyTuple_SET_ITEM(both, 0, first);
    PyTuple_SET_ITEM(both, 1, second);
    return both;
    END_HANDLE_TH_ERRORS
}

// rope_append(q, k, v, k_cache, v_cache, q_start, kv_len, block_table, inv_freq, positions | None, interleaved,
// scale, q_out | None) -> q_out
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    double scale = 0;
    const int interleaved = n_args == 13 ? truth(a[10]) : -1;
    if (interleaved < 0 || !number(a[11], &scale)) Py_RETURN_NONE;
    Call c;
    fd_heads qh{}, kh{}, vh{}, qo{};
    fd_paged_cache cache{};
    fd_paged_batch batch{};
    const at::Tensor *q = c.heads(a[0], &qh, -1, -1, -1);
    if (!q) Py_RETURN_NONE;
    const int64_t n = q->size(0), d = q->size(2);
    c.cache(a[3], a[4], &cache);
    if (!c.ok || cache.head_dim != d) Py_RETURN_NONE;
    c.heads(a[1], &kh, n, cache.kv_heads, d);
    if (c.ok) c.heads(a[2], &vh, n, cache.kv_heads, d);
    int64_t pairs = 0;
    const void *freq = c.ok ? c.flat(a[8], at::kDouble, -1, &pairs) : nullptr;
    if (c.ok) c.batch(a[5], a[6], a[7], n, n, &batch);
    const void *pos = c.ok && a[9] != Py_None ? c.flat(a[9], at::kInt, n) : nullptr;
    if (!c.ok || pairs < 1 || pairs > d / 2) Py_RETURN_NONE;
    const at::Tensor q_out = c.output(a[12], *q, &qo);
    if (!c.ok) Py_RETURN_NONE;
    int st;
    const fd_stream_t stream = c.stream();
    Py_BEGIN_ALLOW_THREADS;
    st = g_append(&qh, &kh, &vh, &qo, &cache, &batch, static_cast<const int *>(pos), static_cast<const double *>(freq),
                  (int)(2 * pairs), interleaved, (float)scale, stream);
    Py_END_ALLOW_THREADS;
    return st ? PyLong_FromLong(st) : wrap(a[12], q_out);
    END_HANDLE_TH_ERRORS
}

// paged_attention(q, k_cache, v_cache, q_start, kv_len, block_table, max_q, scratch, scale | None, causal, window,
// softcap, out | None, lse | None) -> out
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    double scale = 0, softcap = 0;
    int64_t max_q = 0, window = 0, bytes = 0;
    const int causal = n_args == 14 ? truth(a[9]) : -1;
    if (causal < 0 || !whole(a[6], &max_q) || !whole(a[10], &window) || !number(a[11], &softcap) ||
        (a[8] != Py_None && !number(a[8], &scale)) || max_q < 0 || window < 0 || (softcap != 0 && (float)softcap == 0))
        Py_RETURN_NONE;
    Call c;
    fd_heads qh{}, oh{};
    fd_paged_cache cache{};
    fd_paged_batch batch{};
    const at::Tensor *q = c.heads(a[0], &qh, -1, -1, -1);
    if (!q) Py_RETURN_NONE;
    const int64_t n = q->size(0), h = q->size(1), d = q->size(2);
    c.cache(a[1], a[2], &cache);
    if (!c.ok || cache.head_dim != d || cache.kv_heads == 0 || h % cache.kv_heads != 0) Py_RETURN_NONE;
    c.batch(a[3], a[4], a[5], n, max_q < n ? max_q : n, &batch);
    void *scratch = c.ok ? c.flat(a[7], at::kByte, -1, &bytes) : nullptr;
    float *lse = nullptr;
    if (c.ok && a[13] != Py_None) {
        const at::Tensor *t = c.take(a[13], at::kFloat, 2);
        c.ok = t && t->size(0) == n && t->size(1) == h && t->is_contiguous();
        if (c.ok) lse = static_cast<float *>(t->data_ptr());
    }
    if (!c.ok) Py_RETURN_NONE;
    const at::Tensor out = c.output(a[12], *q, &oh);
    if (!c.ok) Py_RETURN_NONE;
    if (a[8] == Py_None) scale = 1.0 / std::sqrt((double)d);
    int st;
    const fd_stream_t stream = c.stream();
    Py_BEGIN_ALLOW_THREADS;
    st = g_attention(&qh, &cache, &batch, &oh, lse, (float)scale, causal, (int)(window < INT32_MAX ? window : INT32_MAX),
                     (float)softcap, scratch, (size_t)bytes, stream);
    Py_END_ALLOW_THREADS;
    return st ? PyLong_FromLong(st) : wrap(a[12], out);
    END_HANDLE_TH_ERRORS
}

// init(addresses of fd_rope, fd_rope_append, fd_paged_attention)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    if (n_args != 3) {
        PyErr_SetString(PyExc_TypeError, "init takes three addresses");
        return nullptr;
    }
    void *p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
    g_append = reinterpret_cast<decltype(g_append)>(p[1]);
    g_attention = reinterpret_cast<decltype(g_attention)>(p[2]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fd_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

#define FD_TEXT_OF(x) #x
#define FD_TEXT(x) FD_TEXT_OF(x)

// `torch_version`, `python_version`: whose headers this was built against (their objects are used as they
// lie in memory).
PyMODINIT_FUNC PyInit__fd_torch() {
    PyObject *m = PyModule_Create(&module);
    if (m && (PyModule_AddStringConstant(m, "torch_version", FD_TORCH_VERSION) < 0 ||
              PyModule_AddStringConstant(m, "python_version",
                                         FD_TEXT(PY_MAJOR_VERSION) "." FD_TEXT(PY_MINOR_VERSION)) < 0))
        Py_CLEAR(m);
    return m;
}
