// _ffn.so: the binding of the feed-forward operators as a CPython module on torch's C++ tensors (the
// paged operators' manner: arguments checked and marshalled here, then the C ABI of include/qaff.h).
#include "marshal.h"

#include <torch/csrc/Dtype.h>

#include <vector>

namespace {

constexpr at::ScalarType kF8 = at::kFloat8_e4m3fn;

bool is_float(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16 || t == at::kHalf; }
qaff_dtype code_of(at::ScalarType t) { return t == at::kFloat ? QAFF_F32 : t == at::kHalf ? QAFF_F16 : QAFF_BF16; }

// A GPU tensor of float32, bf16 or float16.
const at::Tensor& float_tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + " must be on a GPU device, got " + t.device().str());
    if (!is_float(t.scalar_type()))
        raise(PyExc_TypeError, std::string(name) + " has dtype " + type_name(t.scalar_type()) +
                                   ", expected float32, bfloat16 or float16");
    return t;
}

// [..., cols] as rows: how many, and how far apart. A 2-D tensor may have any row stride.
struct Rows {
    int64_t rows, cols, stride;
};
Rows rows_of(const at::Tensor& t, const char* name) {
    if (t.dim() < 1) raise(PyExc_ValueError, std::string(name) + " must have at least one dimension");
    const int64_t cols = t.size(-1);
    int64_t rows = 1;
    for (int64_t i = 0; i + 1 < t.dim(); ++i) rows *= t.size(i);
    if (t.numel() && cols > 1 && t.stride(-1) != 1)
        raise(PyExc_ValueError, std::string("the last axis of ") + name + " must be contiguous");
    if (t.dim() == 2) return {rows, cols, rows > 1 ? t.stride(0) : cols};
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous (or 2-D)");
    return {rows, cols, cols};
}

std::vector<int64_t> with_last(const at::Tensor& t, int64_t last) {
    std::vector<int64_t> s = t.sizes().vec();
    s.back() = last;
    return s;
}

at::Tensor output_of(PyObject* o, const at::Tensor& like, at::IntArrayRef sizes, at::ScalarType type) {
    if (o == Py_None) return empty(sizes, like, type);
    const at::Tensor& t = flat(o, "out", type, &like, -1);
    if (t.sizes() != sizes) raise(PyExc_ValueError, "out has the wrong shape " + shape_of(t));
    return t;
}

PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& logits = float_tensor(a[0], "logits");
        const Rows r = rows_of(logits, "logits");
        const int64_t top_k = integer(a[1], "top_k");
        const float* bias = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor& b = flat(a[2], "bias", at::kFloat, &logits, 1);
            if (b.size(0) != r.cols)
                raise(PyExc_ValueError, "bias must be [" + std::to_string(r.cols) + "], got " + shape_of(b));
            bias = ptr<float>(b);
        }
        const bool sigmoid = truth(a[3]), renormalize = truth(a[4]);
        const double scale = PyFloat_AsDouble(a[5]);
        if (scale == -1.0 && PyErr_Occurred()) throw PyError();
        if (top_k < 0 || top_k > r.cols)
            raise(PyExc_ValueError, "top_k is " + std::to_string(top_k) + " of " + std::to_string(r.cols) + " experts");
        const Place place(logits);
        const std::vector<int64_t> sizes = with_last(logits, top_k);
        const at::Tensor weights = empty(sizes, logits, at::kFloat), chosen = empty(sizes, logits, at::kInt);
        check(qaff_moe_route(ptr<void>(logits), code_of(logits.scalar_type()), r.rows, r.cols, r.stride, bias, sigmoid,
                             top_k, renormalize, (float)scale, ptr<float>(weights), ptr<int32_t>(chosen), place.stream));
        return tuple({weights, chosen});
    });
}

struct Expert {
    const at::Tensor &packed, &scales, &biases;
};

// (packed [experts, rows, cols * bits / 32], scales and biases [experts, rows, cols / group]) of x's type.
Expert expert_weight(PyObject* o, const char* name, const at::Tensor& x, int64_t rows, int64_t cols, int64_t group,
                     int64_t bits, int64_t* experts) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3)
        raise(PyExc_TypeError, std::string(name) + " must be a tuple (packed, scales, biases)");
    const std::string n(name);
    const Expert w{tensor(PyTuple_GET_ITEM(o, 0), (n + " codes").c_str(), at::kInt, at::kUInt32, &x, 3),
                   flat(PyTuple_GET_ITEM(o, 1), (n + " scales").c_str(), x.scalar_type(), &x, 3),
                   flat(PyTuple_GET_ITEM(o, 2), (n + " biases").c_str(), x.scalar_type(), &x, 3)};
    if (!w.packed.is_contiguous()) raise(PyExc_ValueError, n + " codes must be contiguous");
    if (*experts < 0) *experts = w.packed.size(0);
    const int64_t codes[3] = {*experts, rows, cols * bits / 32}, groups[3] = {*experts, rows, cols / group};
    if (w.packed.sizes() != at::IntArrayRef(codes) || w.scales.sizes() != at::IntArrayRef(groups) ||
        w.biases.sizes() != at::IntArrayRef(groups))
        raise(PyExc_ValueError, n + " must be " + std::to_string(*experts) + " experts of [" + std::to_string(rows) + ", " +
                                    std::to_string(cols) + "], got codes " + shape_of(w.packed) + ", scales " +
                                    shape_of(w.scales) + " and biases " + shape_of(w.biases));
    return w;
}

PyObject* moe_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor& x = tensor(a[0], "x", at::kBFloat16, at::kHalf, nullptr, -1);
        const Rows r = rows_of(x, "x");
        if (!x.is_contiguous()) raise(PyExc_ValueError, "x must be contiguous");
        const at::Tensor& chosen = flat(a[1], "experts", at::kInt, &x, -1);
        const at::Tensor& weights = flat(a[2], "weights", at::kFloat, &x, -1);
        if (chosen.dim() != x.dim() || chosen.sizes().slice(0, x.dim() - 1) != x.sizes().slice(0, x.dim() - 1) ||
            weights.sizes() != chosen.sizes())
            raise(PyExc_ValueError, "experts and weights must have x's leading shape and one more axis: x " + shape_of(x) +
                                        ", experts " + shape_of(chosen) + ", weights " + shape_of(weights));
        const int64_t group = integer(a[6], "group_size"), bits = integer(a[7], "bits");
        if (group != 32 && group != 64 && group != 128)
            raise(PyExc_ValueError, "group size " + std::to_string(group) + " is not supported (32, 64 or 128)");
        if (bits < 1 || bits > 8 || bits == 7)
            raise(PyExc_ValueError, std::to_string(bits) + " bits are not supported (1, 2, 3, 4, 5, 6 or 8)");
        if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 3)
            raise(PyExc_TypeError, "gate must be a tuple (packed, scales, biases)");
        const int64_t hidden =
            tensor(PyTuple_GET_ITEM(a[3], 0), "gate codes", at::kInt, at::kUInt32, &x, 3).size(1);
        int64_t experts = -1;
        const Expert gate = expert_weight(a[3], "gate", x, hidden, r.cols, group, bits, &experts);
        const Expert up = expert_weight(a[4], "up", x, hidden, r.cols, group, bits, &experts);
        const Expert down = expert_weight(a[5], "down", x, r.cols, hidden, group, bits, &experts);
        const void* resid = nullptr;
        if (a[8] != Py_None) {
            const at::Tensor& t = flat(a[8], "resid", x.scalar_type(), &x, -1);
            if (t.sizes() != x.sizes()) raise(PyExc_ValueError, "resid must be " + shape_of(x) + ", got " + shape_of(t));
            resid = ptr<void>(t);
        }
        const Place place(x);
        const at::Tensor out = output_of(a[9], x, x.sizes(), x.scalar_type());
        const int64_t top_k = chosen.size(-1);
        const size_t bytes = qaff_moe_ffn_workspace_size(r.rows, r.cols, hidden, top_k, experts, (int32_t)group, (int32_t)bits);
        at::Tensor ws;
        if (bytes) ws = empty({(int64_t)bytes}, x, at::kByte);
        check(qaff_moe_ffn(ptr<void>(x), code_of(x.scalar_type()), r.rows, r.cols, hidden, ptr<int32_t>(chosen),
                           ptr<float>(weights), top_k, experts, ptr<uint32_t>(gate.packed), ptr<void>(gate.scales),
                           ptr<void>(gate.biases), ptr<uint32_t>(up.packed), ptr<void>(up.scales), ptr<void>(up.biases),
                           ptr<uint32_t>(down.packed), ptr<void>(down.scales), ptr<void>(down.biases), (int32_t)group,
                           (int32_t)bits, resid, bytes ? ws.data_ptr() : nullptr, bytes, ptr<void>(out), place.stream));
        return THPVariable_Wrap(out);
    });
}

PyObject* block_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 2, [&] {
        const at::Tensor& x = float_tensor(a[0], "x");
        const Rows r = rows_of(x, "x");
        const int64_t block_rows = integer(a[1], "block_rows");
        if (block_rows != 1 && block_rows != 128)
            raise(PyExc_ValueError, "block_rows is " + std::to_string(block_rows) + " (1 or 128)");
        if (block_rows == 128 && x.dim() != 2) raise(PyExc_ValueError, "blocks of 128 rows take a 2-D x, got " + shape_of(x));
        const Place place(x);
        const at::Tensor codes = empty(x.sizes(), x, kF8);
        std::vector<int64_t> sizes = with_last(x, (r.cols + 127) / 128);
        if (block_rows == 128) sizes[0] = (r.rows + 127) / 128;
        const at::Tensor scales = empty(sizes, x, at::kFloat);
        check(qaff_block_quantize(ptr<void>(x), code_of(x.scalar_type()), r.rows, r.cols, r.stride, (int32_t)block_rows,
                                  ptr<uint8_t>(codes), ptr<float>(scales), place.stream));
        return tuple({codes, scales});
    });
}

PyObject* block_qmm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 6, [&] {
        const at::Tensor& x = flat(a[0], "x", kF8, nullptr, -1);
        const at::Tensor& xs = flat(a[1], "x_scales", at::kFloat, &x, -1);
        const at::Tensor& w = flat(a[2], "w", kF8, &x, 2);
        const at::Tensor& ws = flat(a[3], "w_scales", at::kFloat, &x, 2);
        if (!THPDtype_Check(a[4])) raise(PyExc_TypeError, "out_dtype must be a torch.dtype");
        const at::ScalarType type = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
        if (!is_float(type)) raise(PyExc_TypeError, "out_dtype must be float32, bfloat16 or float16");
        const Rows r = rows_of(x, "x");
        const int64_t rows = w.size(0), kb = (r.cols + 127) / 128;
        const int64_t w_groups[2] = {(rows + 127) / 128, kb};
        if (w.size(1) != r.cols)
            raise(PyExc_ValueError, "x has " + std::to_string(r.cols) + " columns, the weight " + std::to_string(w.size(1)));
        if (xs.sizes() != at::IntArrayRef(with_last(x, kb)) || ws.sizes() != at::IntArrayRef(w_groups))
            raise(PyExc_ValueError, "x " + shape_of(x) + " and w " + shape_of(w) + " need a scale for each 128 columns (and 128 rows "
                                    "of w), got " + shape_of(xs) + " and " + shape_of(ws));
        const Place place(x);
        const at::Tensor out = output_of(a[5], x, with_last(x, rows), type);
        check(qaff_block_qmm(ptr<uint8_t>(x), ptr<float>(xs), r.rows, ptr<uint8_t>(w), ptr<float>(ws), rows, r.cols,
                             ptr<void>(out), code_of(type), place.stream));
        return THPVariable_Wrap(out);
    });
}

PyMethodDef methods[] = {
    {"moe_route", (PyCFunction)(void*)moe_route, METH_FASTCALL, nullptr},
    {"moe_ffn", (PyCFunction)(void*)moe_ffn, METH_FASTCALL, nullptr},
    {"block_quantize", (PyCFunction)(void*)block_quantize, METH_FASTCALL, nullptr},
    {"block_qmm", (PyCFunction)(void*)block_qmm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__ffn() { return PyModule_Create(&module); }
