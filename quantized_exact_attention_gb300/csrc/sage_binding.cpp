// sage_binding.cpp - CPython module that hands torch tensors to the entries of
// the C ABI that serve from a page cache.
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
decltype(&sage_rope) g_rope = nullptr;
decltype(&sage_cache_append_rope) g_cache_append_rope = nullptr;
decltype(&sage_tree_tables) g_tree_tables = nullptr;
decltype(&sage_attn_paged_tree) g_attn_paged_tree = nullptr;
decltype(&sage_cache_keep) g_cache_keep = nullptr;

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

// Both attention entries.  a: q, o, cache address, cache device, table | None, [mask,] workspace, q_len, kv_len,
// prefix_table, prefix_len (each | None), sm_scale, [causal,] stream | None, with `mask` or else with `causal`.
int attn(PyObject* const* a, bool tree) {
    const at::Tensor &q = tensor(a[0], "q: expected a tensor"), &o = tensor(a[1], "o: expected a tensor");
    const sage_page_cache* c = cache_of(a[2]);
    const at::Tensor* table = tensor_or_none(a[4], "table: expected a tensor");
    const at::Tensor* mask = tree ? &tensor(a[5], "mask: expected a tensor") : nullptr;
    PyObject* const* r = a + (tree ? 6 : 5);
    const at::Tensor& ws = tensor(r[0], "workspace: expected a tensor");
    const at::Tensor *q_len = tensor_or_none(r[1], "q_len: expected a tensor"),
                     *kv_len = tensor_or_none(r[2], "kv_len: expected a tensor"),
                     *ptable = tensor_or_none(r[3], "prefix_table: expected a tensor"),
                     *plen = tensor_or_none(r[4], "prefix_len: expected a tensor");
    const double scale = PyFloat_AsDouble(r[5]);
    const int causal = tree ? 0 : PyObject_IsTrue(r[6]);
    PyObject* stream = r[tree ? 6 : 7];
    if ((scale == -1.0 || causal < 0) && PyErr_Occurred()) throw Refused{nullptr};
    OneDevice d(a[3]);
    const sage_tensor qv = view(q), ov = view(o);
    if (o.sizes() != q.sizes() || q.size(3) != c->D) throw Refused{"q and o are [B, H, Nq, D] with the cache's D"};
    for (const at::Tensor* t : {&q, &o, &ws, table, mask, q_len, kv_len, ptable, plen}) d.add(t);
    d.check();
    const int32_t* tp = ints(table, 2, "table: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
    const int32_t* pp = ints(ptable, 1, "prefix_table: expected a contiguous int32 vector");
    const int32_t* ql = ints(q_len, 1, "q_len: expected a contiguous int32 vector");
    const int32_t* kl = ints(kv_len, 1, "kv_len: expected a contiguous int32 vector");
    const int32_t* pl = ints(plen, 1, "prefix_len: expected a contiguous int32 vector");
    const int64_t B = q.size(0), N = q.size(2);
    count(table, B, "table: expected one row for each request");
    count(q_len, B, "q_len: expected one entry for each request");
    count(kv_len, B, "kv_len: expected one entry for each request");
    count(plen, 1, "prefix_len: expected one entry");
    if (!ws.is_contiguous()) throw Refused{"workspace: expected a contiguous tensor"};
    const int64_t ts = table != nullptr ? table->stride(0) : 0;
    const int W = table != nullptr ? as_int(table->size(1)) : 0, Wp = ptable != nullptr ? as_int(ptable->size(0)) : 0;
    if (!tree)
        return g_attn_paged(&qv, &ov, c, as_int(B), as_int(q.size(1)), as_int(N), ql, tp, ts, W, kl, pp, Wp, pl, (float)scale,
                            causal, ws.data_ptr(), (size_t)ws.nbytes(), stream_of(stream));
    constexpr const char* kMask = "mask: expected an int32 tensor [B, Nq, W] or [Nq, W] with 32 tokens to a word, contiguous along its last dimension";
    const int md = (int)mask->dim();
    if (md != 2 && md != 3) throw Refused{kMask};
    const int32_t* mp = ints(mask, md, kMask);
    if (mask->size(md - 2) != N || mask->size(md - 1) < (N + 31) / 32 || (md == 3 && mask->size(0) != B)) throw Refused{kMask};
    return g_attn_paged_tree(&qv, &ov, c, as_int(B), as_int(q.size(1)), as_int(N), ql, tp, ts, W, kl, pp, Wp, pl, mp,
                             md == 3 ? mask->stride(0) : 0, mask->stride(md - 2), (float)scale, ws.data_ptr(),
                             (size_t)ws.nbytes(), stream_of(stream));
}
// (q, o, cache address, cache device, table | None, workspace, q_len, kv_len,
//  prefix_table, prefix_len (each | None), sm_scale, causal, stream | None)
PyObject* attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return arity(n, 13) ? guarded([&]() -> int { return attn(a, false); }) : nullptr;
}
// (q, o, cache address, cache device, table | None, mask, workspace, q_len, kv_len,
//  prefix_table, prefix_len (each | None), sm_scale, stream | None)
PyObject* attn_paged_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return arity(n, 13) ? guarded([&]() -> int { return attn(a, true); }) : nullptr;
}

// Positions of a [B, .., N, ..] call: int32 [B, N], or [N] for all requests; null for none.
struct Positions {
    const int32_t* at;
    int64_t stride;
};
Positions positions_of(const at::Tensor* t, int64_t B, int64_t N) {
    constexpr const char* kWhat = "positions: expected an int32 tensor [B, N] or [N], contiguous along its last dimension";
    if (t == nullptr) return {nullptr, 0};
    if (t->dim() != 1 && t->dim() != 2) throw Refused{kWhat};
    const int32_t* p = ints(t, (int)t->dim(), kWhat);
    if (t->size(t->dim() - 1) != N || (t->dim() == 2 && t->size(0) != B)) throw Refused{kWhat};
    return {p, t->dim() == 2 ? t->stride(0) : 0};
}
const sage_rotary* rotary_of(PyObject* address, PyObject* device, OneDevice& d) {
    void* r = PyLong_AsVoidPtr(address);
    if (r == nullptr) throw Refused{PyErr_Occurred() ? nullptr : "no rotary positions"};
    const int dev = (int)PyLong_AsLong(device);
    if (dev < 0) throw Refused{PyErr_Occurred() ? nullptr : "the rotary positions live on a CUDA device"};
    if (d.dev < 0) d.dev = dev;
    if (d.dev != dev) throw Refused{"all tensors of a call live on one CUDA device"};
    return static_cast<const sage_rotary*>(r);
}

// (x, out, rotary address, rotary device, positions, start, n_len (each | None), inverse, stream | None)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 9)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &x = tensor(a[0], "x: expected a tensor"), &out = tensor(a[1], "out: expected a tensor");
        const at::Tensor *positions = tensor_or_none(a[4], "positions: expected a tensor"),
                         *start = tensor_or_none(a[5], "start: expected a tensor"),
                         *n_len = tensor_or_none(a[6], "n_len: expected a tensor");
        const int inverse = PyObject_IsTrue(a[7]);
        if (inverse < 0) throw Refused{nullptr};
        const sage_tensor xv = view(x), ov = view(out);
        if (out.sizes() != x.sizes()) throw Refused{"x and out are [B, H, N, D] of one shape"};
        OneDevice d;
        const sage_rotary* r = rotary_of(a[2], a[3], d);
        for (const at::Tensor* t : {&x, &out, positions, start, n_len}) d.add(t);
        d.check();
        const int64_t B = x.size(0), N = x.size(2);
        const Positions at = positions_of(positions, B, N);
        const int32_t* sp = ints(start, 1, "start: expected a contiguous int32 vector");
        const int32_t* np = ints(n_len, 1, "n_len: expected a contiguous int32 vector");
        count(start, B, "start: expected one entry for each request");
        count(n_len, B, "n_len: expected one entry for each request");
        return g_rope(&xv, &ov, as_int(B), as_int(x.size(1)), as_int(N), as_int(x.size(3)), at.at, at.stride, sp, np, r, inverse,
                      stream_of(a[8]));
    });
}

// (k, v, slots, cache address, cache device, rotary address, rotary device, positions, start (each | None), stream | None)
PyObject* cache_append_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 10)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &k = tensor(a[0], "k: expected a tensor"), &v = tensor(a[1], "v: expected a tensor"),
                         &slots = tensor(a[2], "slots: expected a tensor");
        const at::Tensor *positions = tensor_or_none(a[7], "positions: expected a tensor"),
                         *start = tensor_or_none(a[8], "start: expected a tensor");
        const sage_page_cache* c = cache_of(a[3]);
        const sage_tensor kv = view(k), vv = view(v);
        if (v.sizes() != k.sizes() || k.size(1) != c->heads || k.size(3) != c->D)
            throw Refused{"k and v are [B, heads, N, D] with the cache's heads and D"};
        OneDevice d(a[4]);
        const sage_rotary* r = rotary_of(a[5], a[6], d);
        for (const at::Tensor* t : {&k, &v, &slots, positions, start}) d.add(t);
        d.check();
        const int64_t B = k.size(0), N = k.size(2);
        const int32_t* sl = ints(&slots, 2, "slots: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        if (slots.size(0) != B || slots.size(1) != N) throw Refused{"slots: expected [B, N] as of k"};
        const Positions at = positions_of(positions, B, N);
        const int32_t* sp = ints(start, 1, "start: expected a contiguous int32 vector");
        count(start, B, "start: expected one entry for each request");
        return g_cache_append_rope(&kv, &vv, as_int(B), as_int(N), sl, slots.stride(0), at.at, at.stride, sp, r, c,
                                   stream_of(a[9]));
    });
}

// (parents, mask, depth, n_len (each | None), stream | None)
PyObject* tree_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 5)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &parents = tensor(a[0], "parents: expected a tensor"), &mask = tensor(a[1], "mask: expected a tensor");
        const at::Tensor *depth = tensor_or_none(a[2], "depth: expected a tensor"),
                         *n_len = tensor_or_none(a[3], "n_len: expected a tensor");
        OneDevice d;
        for (const at::Tensor* t : {&parents, &mask, depth, n_len}) d.add(t);
        d.check();
        const int32_t* pp =
            ints(&parents, 2, "parents: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        int32_t* mp = ints(&mask, 3, "mask: expected a 3-dimensional int32 tensor, contiguous along its last dimension");
        int32_t* dp = ints(depth, 2, "depth: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        const int32_t* np = ints(n_len, 1, "n_len: expected a contiguous int32 vector");
        const int64_t B = parents.size(0), N = parents.size(1);
        if (mask.size(0) != B || mask.size(1) != N || mask.size(2) < (N + 31) / 32)
            throw Refused{"mask: expected [B, N, W] with 32 tokens to a word"};
        if (depth != nullptr && (depth->size(0) != B || depth->size(1) != N)) throw Refused{"depth: expected [B, N] as of parents"};
        count(n_len, B, "n_len: expected one entry for each request");
        return g_tree_tables(pp, parents.stride(0), as_int(B), as_int(N), np, mp, mask.stride(0), mask.stride(1), dp,
                             depth != nullptr ? depth->stride(0) : 0, stream_of(a[4]));
    });
}

// (kept, slots, cache address, cache device, stream | None)
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 5)) return nullptr;
    return guarded([&]() -> int {
        const at::Tensor &kept = tensor(a[0], "kept: expected a tensor"), &slots = tensor(a[1], "slots: expected a tensor");
        const sage_page_cache* c = cache_of(a[2]);
        OneDevice d(a[3]);
        for (const at::Tensor* t : {&kept, &slots}) d.add(t);
        d.check();
        const int32_t* kp = ints(&kept, 2, "kept: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        const int32_t* sp = ints(&slots, 2, "slots: expected a 2-dimensional int32 tensor, contiguous along its last dimension");
        if (kept.size(0) != slots.size(0) || kept.size(1) > slots.size(1))
            throw Refused{"kept: expected [B, K] with the rows of slots and no more columns"};
        return g_cache_keep(kp, kept.stride(0), as_int(kept.size(0)), as_int(kept.size(1)), sp, slots.stride(0),
                            as_int(slots.size(1)), c, stream_of(a[4]));
    });
}

template <class F>
void take(F& entry, PyObject* address) {
    entry = reinterpret_cast<F>(PyLong_AsVoidPtr(address));
}
// The addresses of the entries, in the order of their declaration above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    take(g_page_tables, a[0]);
    take(g_cache_append, a[1]);
    take(g_attn_paged, a[2]);
    take(g_rope, a[3]);
    take(g_cache_append_rope, a[4]);
    take(g_tree_tables, a[5]);
    take(g_attn_paged_tree, a[6]);
    take(g_cache_keep, a[7]);
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, "Take the entries' addresses."},
    {"page_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(page_tables)), METH_FASTCALL, "sage_page_tables"},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_append)), METH_FASTCALL, "sage_cache_append"},
    {"attn_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn_paged)), METH_FASTCALL, "sage_attn_paged"},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, "sage_rope"},
    {"cache_append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_append_rope)), METH_FASTCALL, "sage_cache_append_rope"},
    {"tree_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(tree_tables)), METH_FASTCALL, "sage_tree_tables"},
    {"attn_paged_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attn_paged_tree)), METH_FASTCALL, "sage_attn_paged_tree"},
    {"cache_keep", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache_keep)), METH_FASTCALL, "sage_cache_keep"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_sage_binding", "Page-cache entries on torch tensors.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sage_binding(void) { return PyModule_Create(&kModule); }
