// _paged.so: the binding of the paged-cache operators as a CPython module on torch's C++ tensors.
//
// It marshals arguments as the ctypes binding does (devices, dtypes, shapes, strides; outputs and
// workspace from torch's allocator; the current stream) and calls the C ABI of include/qaff.h. A
// serving step makes these calls once or thrice per layer with kernels of a few microseconds, so the
// call itself counts: through ctypes and Python checks a call took 15 us, here 5 to 7.
#include "marshal.h"

#include <cmath>

namespace {

// A [tokens, heads, head_dim] operand whose last axis is contiguous.
const at::Tensor& heads_of(PyObject* o, const char* name, at::ScalarType t0, at::ScalarType t1, const at::Tensor* like) {
    const at::Tensor& t = tensor(o, name, t0, t1, like, 3);
    if (t.size(2) > 1 && t.stride(2) != 1)
        raise(PyExc_ValueError, std::string("the last axis of ") + name + " must be contiguous");
    return t;
}

struct Caches {
    const at::Tensor &k, &v;
    int64_t pages, kv_heads, page_size, dim, stride;
};

Caches caches(PyObject* ko, PyObject* vo, const at::Tensor& q) {
    const at::Tensor& k = tensor(ko, "k_cache", q.scalar_type(), q.scalar_type(), &q, 4);
    const at::Tensor& v = tensor(vo, "v_cache", q.scalar_type(), q.scalar_type(), &q, 4);
    if (k.sizes() != v.sizes())
        raise(PyExc_ValueError, "k_cache " + shape_of(k) + " and v_cache " + shape_of(v) + " differ");
    Caches c{k, v, k.size(0), k.size(1), k.size(2), k.size(3), k.stride(0)};
    // an axis of size 1 may have any stride
    auto stride_is = [](const at::Tensor& t, int64_t axis, int64_t stride) {
        return t.size(axis) <= 1 || t.stride(axis) == stride;
    };
    for (const at::Tensor* t : {&k, &v})
        if (t->numel() && !(stride_is(*t, 1, c.page_size * c.dim) && stride_is(*t, 2, c.dim) && stride_is(*t, 3, 1)))
            raise(PyExc_ValueError, "each page of the caches must be contiguous: [kv_heads, page_size, head_dim]");
    if (k.numel() && !stride_is(v, 0, c.stride)) raise(PyExc_ValueError, "k_cache and v_cache differ in their strides");
    if (c.pages <= 1) c.stride = c.kv_heads * c.page_size * c.dim;
    return c;
}

// n values of `type` from byte `at` of a buffer on, as a tensor of their own that shares the buffer:
// a tenth of the time of another allocation.
at::Tensor piece(const at::Tensor& buffer, int64_t at, int64_t n, at::ScalarType type) {
    auto t = c10::make_intrusive<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(),
                                                  c10::scalarTypeToTypeMeta(type));
    t->set_sizes_contiguous({n});
    t->set_storage_offset(at / (int64_t)c10::elementSize(type));
    return at::Tensor(std::move(t));
}

// The output: `o`, checked, or a new tensor of q's shape.
at::Tensor output(PyObject* o, const at::Tensor& q) {
    if (o == Py_None) return empty(q.sizes(), q, q.scalar_type());
    const at::Tensor& t = flat(o, "out", q.scalar_type(), &q, 3);
    if (t.sizes() != q.sizes()) raise(PyExc_ValueError, "out must be " + shape_of(q));
    return t;
}

PyObject* paged_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& cached = flat(a[0], "cached_lens", at::kInt, nullptr, 1);
        const at::Tensor& fresh = flat(a[1], "new_lens", at::kInt, &cached, 1);
        const at::Tensor& free_pages = flat(a[2], "free_pages", at::kInt, &cached, 1);
        const at::Tensor& tables = flat(a[3], "block_tables", at::kInt, &cached, 2);
        const int64_t page_size = integer(a[4], "page_size"), tokens = integer(a[5], "tokens");
        const int64_t requests = cached.size(0);
        if (fresh.size(0) != requests || tables.size(0) != requests)
            raise(PyExc_ValueError, "cached_lens has " + std::to_string(requests) + " requests, new_lens " +
                                        std::to_string(fresh.size(0)) + ", block_tables " + std::to_string(tables.size(0)));
        if (tokens < 0) raise(PyExc_ValueError, "tokens is " + std::to_string(tokens));
        const Place place(cached);
        // one buffer for the five outputs: slots, then the int32 ones
        if (tokens >= (int64_t)1 << 31) raise(PyExc_ValueError, "tokens is " + std::to_string(tokens) + ", 2^31 or more");
        const int64_t at_cu = 8 * tokens, at_kv = at_cu + 4 * (requests + 1), at_pos = at_kv + 4 * requests,
                      at_used = at_pos + 4 * tokens;
        const at::Tensor all = empty({at_used / 8 + 1}, cached, at::kLong);
        const at::Tensor cu = piece(all, at_cu, requests + 1, at::kInt), kv = piece(all, at_kv, requests, at::kInt),
                         positions = piece(all, at_pos, tokens, at::kInt), slots = piece(all, 0, tokens, at::kLong),
                         used = piece(all, at_used, 1, at::kInt);
        check(qaff_paged_plan(ptr<int32_t>(cached), ptr<int32_t>(fresh), requests, ptr<int32_t>(free_pages),
                              free_pages.size(0), ptr<int32_t>(tables), tables.size(1),
                              page_size == (int32_t)page_size ? (int32_t)page_size : -1, tokens, ptr<int32_t>(cu),
                              ptr<int32_t>(kv), ptr<int32_t>(positions), ptr<int64_t>(slots), ptr<int32_t>(used),
                              place.stream));
        return tuple({cu, kv, positions, slots, used});
    });
}

PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor& q = heads_of(a[0], "q", at::kBFloat16, at::kHalf, nullptr);
        const at::Tensor& k = heads_of(a[1], "k", q.scalar_type(), q.scalar_type(), &q);
        const at::Tensor& v = heads_of(a[2], "v", q.scalar_type(), q.scalar_type(), &q);
        const at::Tensor& positions = flat(a[3], "positions", at::kInt, &q, -1);
        const at::Tensor& inv_freq = flat(a[4], "inv_freq", at::kFloat, &q, 1);
        const at::Tensor& slots = flat(a[5], "slots", at::kLong, &q, 1);
        const Caches c = caches(a[6], a[7], q);
        const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
        const int64_t want[3] = {tokens, c.kv_heads, dim};
        if (c.dim != dim || k.sizes() != at::IntArrayRef(want) || v.sizes() != at::IntArrayRef(want))
            raise(PyExc_ValueError, "q " + shape_of(q) + " with caches " + shape_of(c.k) + " needs k and v [" +
                                        std::to_string(tokens) + ", " + std::to_string(c.kv_heads) + ", " +
                                        std::to_string(dim) + "], got " + shape_of(k) + " and " + shape_of(v));
        if (positions.dim() < 1 || positions.dim() > 2 || positions.size(-1) != tokens)
            raise(PyExc_ValueError, "positions must be [" + std::to_string(tokens) + "] or [axes, " +
                                        std::to_string(tokens) + "], got " + shape_of(positions));
        const int64_t axes = positions.dim() == 1 ? 1 : positions.size(0);
        if (slots.size(0) != tokens)
            raise(PyExc_ValueError, "slots must be [" + std::to_string(tokens) + "], got " + shape_of(slots));
        int32_t sections[4] = {0, 0, 0, 0};
        if (a[8] != Py_None) {
            PyObject* seq = PySequence_Fast(a[8], "sections must be a sequence");
            if (!seq) throw PyError();
            const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
            bool fits = count == axes && count <= 4;
            for (Py_ssize_t i = 0; fits && i < count; ++i) {
                const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
                if (v == -1 && PyErr_Occurred()) {
                    Py_DECREF(seq);
                    throw PyError();
                }
                sections[i] = v < 0 || v > (1 << 20) ? -1 : (int32_t)v;
            }
            Py_DECREF(seq);
            if (!fits)
                raise(PyExc_ValueError, std::to_string(count) + " sections for " + std::to_string(axes) + " axes (1 to 4)");
        }
        const bool interleaved = truth(a[9]), traditional = truth(a[10]);
        const Place place(q);
        const at::Tensor out = output(a[11], q);
        check(qaff_rope_append(ptr<void>(q), ptr<void>(k), ptr<void>(v), dtype_of(q), tokens, heads, c.kv_heads, dim,
                               q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                               ptr<int32_t>(positions), (int32_t)std::min<int64_t>(axes, 5),
                               a[8] == Py_None ? nullptr : sections, interleaved, traditional, ptr<float>(inv_freq),
                               2 * inv_freq.size(0), ptr<int64_t>(slots), ptr<void>(c.k), ptr<void>(c.v), c.pages,
                               c.stride, (int32_t)std::min<int64_t>(c.page_size, 1 << 20), ptr<void>(out), place.stream));
        return THPVariable_Wrap(out);
    });
}

PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor& q = heads_of(a[0], "q", at::kBFloat16, at::kHalf, nullptr);
        const Caches c = caches(a[1], a[2], q);
        const at::Tensor& tables = flat(a[3], "block_tables", at::kInt, &q, 2);
        const at::Tensor& cu = flat(a[4], "cu_new", at::kInt, &q, 1);
        const at::Tensor& kv = flat(a[5], "kv_lens", at::kInt, &q, 1);
        const int64_t tokens = q.size(0), heads = q.size(1), dim = q.size(2);
        const int64_t requests = tables.size(0), width = tables.size(1);
        if (c.dim != dim)
            raise(PyExc_ValueError, "q has heads of " + std::to_string(dim) + ", the caches of " + std::to_string(c.dim));
        if (kv.size(0) != requests || cu.size(0) != requests + 1)
            raise(PyExc_ValueError, "block_tables has " + std::to_string(requests) + " requests, kv_lens " +
                                        std::to_string(kv.size(0)) + ", cu_new needs " + std::to_string(requests + 1) +
                                        " entries and has " + std::to_string(cu.size(0)));
        const int64_t max_new = a[6] == Py_None ? tokens : integer(a[6], "max_new");
        double scale = dim ? 1.0 / std::sqrt((double)dim) : 1.0;
        if (a[7] != Py_None) {
            scale = PyFloat_AsDouble(a[7]);
            if (scale == -1.0 && PyErr_Occurred()) throw PyError();
        }
        const bool causal = truth(a[8]), with_lse = truth(a[10]);
        const int64_t window = integer(a[9], "window");
        const int32_t page_size = (int32_t)std::min<int64_t>(c.page_size, 1 << 20);
        const Place place(q);
        const at::Tensor out = output(a[11], q);
        at::Tensor lse, ws;
        if (with_lse) lse = empty({tokens, heads}, q, at::kFloat);
        const size_t bytes = qaff_paged_attention_workspace_size(tokens, heads, c.kv_heads, dim, page_size, width, requests,
                                                                 max_new);
        if (bytes) ws = empty({(int64_t)bytes}, q, at::kByte);
        check(qaff_paged_attention(ptr<void>(q), dtype_of(q), tokens, heads, q.stride(0), q.stride(1), ptr<void>(c.k),
                                   ptr<void>(c.v), c.pages, c.stride, c.kv_heads, dim, page_size, ptr<int32_t>(tables),
                                   width, ptr<int32_t>(cu), ptr<int32_t>(kv), requests, max_new, (float)scale, causal,
                                   window, bytes ? ws.data_ptr() : nullptr, bytes, ptr<void>(out),
                                   with_lse ? ptr<float>(lse) : nullptr, place.stream));
        return with_lse ? tuple({out, lse}) : THPVariable_Wrap(out);
    });
}

PyMethodDef methods[] = {
    {"paged_plan", (PyCFunction)(void*)paged_plan, METH_FASTCALL, nullptr},
    {"rope_append", (PyCFunction)(void*)rope_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void*)paged_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__paged() { return PyModule_Create(&module); }
