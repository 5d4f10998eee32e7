// sage_binding.cpp - CPython module that hands torch tensors to the page-cache
// entries of the C ABI.
//
// A serving loop makes these calls once per layer and token, so their host
// time is part of their latency: reading a tensor's attributes from Python
// costs about 0.1 us each, 6 us in all for a call with seven tensors; here it
// is a few loads.  The module only checks and marshals; the entries are the
// library's, given to it as addresses by the package that loaded the library.
// Argument errors raise ValueError; a C status is returned as it is.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sage_gb300.h"

namespace {

decltype(&sage_page_tables) g_page_tables = nullptr;
decltype(&sage_cache_append) g_cache_append = nullptr;
decltype(&sage_attn_paged) g_attn_paged = nullptr;

// Thrown for an argument the call refuses.
struct Refused {
    const char* what;
};

const at::Tensor* tensor_or_none(PyObject* o, const char* what) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) throw Refused{what};
    return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* what) {
    const at::Tensor* t = tensor_or_none(o, what);
    if (t == nullptr) throw Refused{what};
    return *t;
}

// All tensors of a call live on the current CUDA device.
struct OneDevice {
    int dev = -1;                                       // -1: taken from the first tensor
    OneDevice() = default;
    explicit OneDevice(PyObject* cache_device) : dev((int)PyLong_AsLong(cache_device)) {
        if (dev < 0) throw Refused{PyErr_Occurred() ? nullptr : "the page cache lives on a CUDA device"};
    }
    void add(const at::Tensor* t) {
        if (t == nullptr) return;
        if (!t->is_cuda()) throw Refused{"the tensors of a call live on a CUDA device"};
        const int d = t->get_device();
        if (dev < 0) dev = d;
        if (d != dev) throw Refused{"all tensors of a call live on one CUDA device"};
    }
    void check() const {
        if (c10::cuda::current_device() != dev) throw Refused{"the tensors of a call live on the current CUDA device"};
    }
};

// int32, `dim` dimensions, contiguous along the last; null for none.
int32_t* ints(const at::Tensor* t, int dim, const char* what) {
    if (t == nullptr) return nullptr;
    if (t->scalar_type() != at::kInt || t->dim() != dim || (t->size(dim - 1) > 1 && t->stride(dim - 1) != 1))
        throw Refused{what};
    return static_cast<int32_t*>(t->data_ptr());
}
void count(const at::Tensor* t, int64_t n, const char* what) {
    if (t != nullptr && t->size(0) != n) throw Refused{what};
}
int as_int(int64_t n) {
    if (n > INT32_MAX) throw Refused{"a size passes 2^31 - 1"};
    return static_cast<int>(n);
}

sage_tensor view(const at::Tensor& t) {
    if (t.dim() != 4 || t.scalar_type() != at::kBFloat16 || (t.size(3) > 1 && t.stride(3) != 1))
        throw Refused{"expected a [B, H, N, D] bfloat16 view with unit D stride"};
    return sage_tensor{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
}

void* stream_of(PyObject* o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* s = PyLong_AsVoidPtr(o);
    if (s == nullptr && PyErr_Occurred()) throw Refused{nullptr};
    return s;
}
const sage_page_cache* cache_of(PyObject* o) {
    void* c = PyLong_AsVoidPtr(o);
    if (c == nullptr) throw Refused{PyErr_Occurred() ? nullptr : "no page cache"};
    return static_cast<const sage_page_cache*>(c);
}

// The body of an entry: its status as a Python int, or an exception.
template <class F>
PyObject* guarded(F&& f) {
    try {
        return PyLong_FromLong(f());
    } catch (const Refused& r) {
        if (r.what != nullptr) PyErr_SetString(PyExc_ValueError, r.what);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}
bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// (new_len, page_size, free_pages, table, slots | None, taken, old_len | None, stream | None)
PyObject* page_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &new_len = tensor(a[0], "new_len: expected a tensor"),
                         &free_pages = tensor(a[2], "free_pages: expected a tensor"),
                         &table = tensor(a[3], "table: expected a tensor"), &taken = tensor(a[5], "taken: expected a tensor");
        const at::Tensor *slots = tensor_or_none(a[4], "slots: expected a tensor"),
                         *old_len = tensor_or_none(a[6], "old_len: expected a tensor");
        const long page = PyLong_AsLong(a[1]);
        if (page == -1 && PyErr_Occurred()) throw Refused{nullptr};
        if (page < 0 || page > INT32_MAX) throw Refused{"page_size: expected 16, 32, 64 or 128"};
        OneDevice d;
        for (const at::Tensor* t : {&table, &new_len, &free_pages, &taken, slots, old_len}) d.add(t);
        d.check();
        int32_t* tp = ints(&table, 2, "table: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        int32_t* sp = ints(slots, 2, "slots: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        const int32_t* np = ints(&new_len, 1, "new_len: expected a contiguous int32 vector");
        const int32_t* op = ints(old_len, 1, "old_len: expected a contiguous int32 vector");
        const int32_t* fp = ints(&free_pages, 1, "free_pages: expected a contiguous int32 vector");
        int32_t* kp = ints(&taken, 1, "taken: expected a contiguous int32 vector");
        const int64_t B = table.size(0);
        count(&new_len, B, "new_len: expected one entry for each row of the table");
        count(old_len, B, "old_len: expected one entry for each row of the table");
        count(slots, B, "slots: expected one row for each row of the table");
        count(&taken, 1, "taken: expected one entry");
        return g_page_tables(op, np, as_int(B), (int)page, fp, as_int(free_pages.size(0)), tp, table.stride(0),
                             as_int(table.size(1)), sp, slots != nullptr ? slots->stride(0) : 0,
                             slots != nullptr ? as_int(slots->size(1)) : 0, kp, stream_of(a[7]));
    });
}

// (k, v, slots, cache address, cache device, stream | None)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 6)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &k = tensor(a[0], "k: expected a tensor"), &v = tensor(a[1], "v: expected a tensor"),
                         &slots = tensor(a[2], "slots: expected a tensor");
        const sage_page_cache* c = cache_of(a[3]);
        OneDevice d(a[4]);
        const sage_tensor kv = view(k), vv = view(v);
        if (v.sizes() != k.sizes() || k.size(1) != c->heads || k.size(3) != c->D)
            throw Refused{"k and v are [B, heads, N, D] with the cache's heads and D"};
        for (const at::Tensor* t : {&k, &v, &slots}) d.add(t);
        d.check();
        const int32_t* sp = ints(&slots, 2, "slots: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        if (slots.size(0) != k.size(0) || slots.size(1) != k.size(2)) throw Refused{"slots: expected [B, N] as of k"};
        return g_cache_append(&kv, &vv, as_int(k.size(0)), as_int(k.size(2)), sp, slots.stride(0), c, stream_of(a[5]));
    });
}

// (q, o, cache address, cache device, table | None, workspace, q_len, kv_len,
//  prefix_table, prefix_len (each | None), sm_scale, causal, stream | None)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 13)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &q = tensor(a[0], "q: expected a tensor"), &o = tensor(a[1], "o: expected a tensor"),
                         &ws = tensor(a[5], "workspace: expected a tensor");
        const sage_page_cache* c = cache_of(a[2]);
        const at::Tensor *table = tensor_or_none(a[4], "table: expected a tensor"),
                         *q_len = tensor_or_none(a[6], "q_len: expected a tensor"),
                         *kv_len = tensor_or_none(a[7], "kv_len: expected a tensor"),
                         *ptable = tensor_or_none(a[8], "prefix_table: expected a tensor"),
                         *plen = tensor_or_none(a[9], "prefix_len: expected a tensor");
        const double scale = PyFloat_AsDouble(a[10]);
        const int causal = PyObject_IsTrue(a[11]);
        if ((scale == -1.0 || causal < 0) && PyErr_Occurred()) throw Refused{nullptr};
        OneDevice d(a[3]);
        const sage_tensor qv = view(q), ov = view(o);
        if (o.sizes() != q.sizes() || q.size(3) != c->D) throw Refused{"q and o are [B, H, Nq, D] with the cache's D"};
        for (const at::Tensor* t : {&q, &o, &ws, table, q_len, kv_len, ptable, plen}) d.add(t);
        d.check();
        const int32_t* tp = ints(table, 2, "table: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        const int32_t* pp = ints(ptable, 1, "prefix_table: expected a contiguous int32 vector");
        const int32_t* ql = ints(q_len, 1, "q_len: expected a contiguous int32 vector");
        const int32_t* kl = ints(kv_len, 1, "kv_len: expected a contiguous int32 vector");
        const int32_t* pl = ints(plen, 1, "prefix_len: expected a contiguous int32 vector");
        const int64_t B = q.size(0);
        count(table, B, "table: expected one row for each request");
        count(q_len, B, "q_len: expected one entry for each request");
        count(kv_len, B, "kv_len: expected one entry for each request");
        count(plen, 1, "prefix_len: expected one entry");
        if (!ws.is_contiguous()) throw Refused{"workspace: expected a contiguous tensor"};
        return g_attn_paged(&qv, &ov, c, as_int(B), as_int(q.size(1)), as_int(q.size(2)), ql, tp,
                            table != nullptr ? table->stride(0) : 0, table != nullptr ? as_int(table->size(1)) : 0, kl, pp,
                            ptable != nullptr ? as_int(ptable->size(0)) : 0, pl, (float)scale, causal, ws.data_ptr(),
                            (size_t)ws.nbytes(), stream_of(a[12]));
    });
}

// (address of sage_page_tables, of sage_cache_append, of sage_attn_paged)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 3)) return nullptr;
    g_page_tables = reinterpret_cast<decltype(g_page_tables)>(PyLong_AsVoidPtr(a[0]));
    g_cache_append = reinterpret_cast<decltype(g_cache_append)>(PyLong_AsVoidPtr(a[1]));
    g_attn_paged = reinterpret_cast<decltype(g_attn_paged)>(PyLong_AsVoidPtr(a[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, "Take the entries' addresses."},
    {"page_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_tables)), METH_FASTCALL, "sage_page_tables"},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_append)), METH_FASTCALL, "sage_cache_append"},
    {"attn_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn_paged)), METH_FASTCALL, "sage_attn_paged"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sage_binding", "Page-cache entries on torch tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sage_binding(void) { return PyModule_Create(&kModule); }
