// zc_experts_binding.cpp -- the expert operators' calls from Python: reads
// tensors, checks them, and calls the C ABI (zc_experts.h).
//
// The kernels of a decoding step take a few microseconds, as long as checking
// a call's tensors from Python would (5.5 us a call, 3.3 of them the library's
// call by ctypes); here both take 2.9.  Argument marshalling and checks only:
// every refusal is a ZcError, and nothing is launched then.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "zc_experts.h"

namespace {

// The library's functions, by the addresses that the Python side found.
struct Library {
    decltype(&zc_route) route;
    decltype(&zc_dispatch) dispatch;
    decltype(&zc_dispatch_fp8) dispatch_fp8;
    decltype(&zc_combine) combine;
    decltype(&zc_combine_backward) combine_backward;
    decltype(&zc_quantize_rows) quantize_rows;
    decltype(&zc_quantize_weights) quantize_weights;
    decltype(&zc_quantize_columns) quantize_columns;
    decltype(&zc_expert_product) expert_product;
    decltype(&zc_expert_weight_grad) expert_weight_grad;
    decltype(&zc_expert_weight_grad_workspace_bytes) expert_weight_grad_workspace_bytes;
} zc;
PyObject* error_type = nullptr;  // binding.ZcError

struct Refused {
    int code;
    std::string what;
};
struct PythonError {};  // already set

[[noreturn]] void refuse(const char* what, const std::string& why, int code = ZC_ERR_INVALID_ARG) {
    throw Refused{code, std::string(what) + ": " + why};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

int dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return ZC_BF16;
        case at::kHalf: return ZC_FP16;
        case at::kFloat: return ZC_FP32;
        default: return -1;
    }
}

uint64_t up(uint64_t n, uint64_t m) { return (n + m - 1) / m * m; }

// A size that the library takes in 32 bits.
uint32_t size32(uint64_t v, const char* what) {
    if (v >> 32) refuse(what, "size " + std::to_string(v), ZC_ERR_UNSUPPORTED);
    return (uint32_t)v;
}

struct Matrix {
    void* p;
    uint64_t stride, rows;
    uint32_t width;
    int dtype;
};

// One call: its tensors have to be on one GPU, the current one.
class Call {
public:
    const at::Tensor& tensor(PyObject* o, const char* what) {
        if (!THPVariable_Check(o)) refuse(what, "not a GPU tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(what, "not a GPU tensor");
        if (device < 0) device = t.get_device();
        else if (device != t.get_device()) refuse(what, "not on the GPU of the other tensors");
        return t;
    }

    // A matrix that is contiguous along its columns, of one of the three row
    // types (dtype < 0) or the given one, with at least `rows` rows and (width
    // >= 0) exactly `width` columns.
    Matrix matrix(PyObject* o, const char* what, uint64_t rows, int dtype = -1, int64_t width = -1) {
        const at::Tensor& t = tensor(o, what);
        const int have = dtype_of(t.scalar_type());
        if (have < 0 || (dtype >= 0 && have != dtype)) refuse(what, std::string("type ") + c10::toString(t.scalar_type()));
        if (t.dim() != 2 || (width >= 0 && t.size(1) != width))
            refuse(what, "shape " + shape_text(t.sizes()) + ", (rows, " + (width < 0 ? "columns" : std::to_string(width)) + ") expected");
        const int64_t n = t.size(0), w = t.size(1);
        int64_t s = t.stride(0);
        if (s < w) {
            if (n > 1) refuse(what, "strides " + shape_text(t.strides()) + ": rows overlap");
            s = w;
        }
        if (t.stride(1) != 1 && w > 1) refuse(what, "strides " + shape_text(t.strides()) + ": columns must be contiguous");
        if ((uint64_t)n < rows) refuse(what, std::to_string(n) + " rows, " + std::to_string(rows) + " needed", ZC_ERR_CAPACITY);
        return Matrix{t.data_ptr(), (uint64_t)s, (uint64_t)n, size32(w, what), have};
    }

    // A contiguous tensor of `type` with at least `count` elements.
    template <typename T = void>
    T* flat(PyObject* o, const char* what, at::ScalarType type, uint64_t count, uint64_t* have = nullptr) {
        const at::Tensor& t = tensor(o, what);
        if (t.scalar_type() != type)
            refuse(what, std::string("type ") + c10::toString(t.scalar_type()) + ", " + c10::toString(type) + " expected");
        if (!t.is_contiguous()) refuse(what, "not contiguous");
        if ((uint64_t)t.numel() < count)
            refuse(what, std::to_string(t.numel()) + " elements, " + std::to_string(count) + " needed", ZC_ERR_CAPACITY);
        if (have) *have = t.numel();
        return static_cast<T*>(t.data_ptr());
    }
    template <typename T = void>
    T* flat_or_null(PyObject* o, const char* what, at::ScalarType type, uint64_t count) {
        return o == Py_None ? nullptr : flat<T>(o, what, type, count);
    }

    // Data or scales of blocks: contiguous, at least lead[0] long, otherwise
    // of shape lead x width.
    uint64_t longest = 0;  // the first dimension of the last one
    void* part(PyObject* o, const char* what, at::ScalarType type, std::initializer_list<uint64_t> lead, uint64_t width) {
        const at::Tensor& t = tensor(o, what);
        if (t.scalar_type() != type)
            refuse(what, std::string("type ") + c10::toString(t.scalar_type()) + ", " + c10::toString(type) + " expected");
        if (!t.is_contiguous()) refuse(what, "not contiguous");
        const uint64_t* l = lead.begin();
        if (t.dim() != (int64_t)lead.size() + 1 || (uint64_t)t.size(-1) != width ||
            (lead.size() > 1 && (uint64_t)t.size(1) != l[1])) {
            std::string want;
            for (uint64_t v : lead) want += std::to_string(v) + ", ";
            refuse(what, "shape " + shape_text(t.sizes()) + ", (" + want + std::to_string(width) + ") expected");
        }
        if ((uint64_t)t.size(0) < l[0])
            refuse(what, std::to_string(t.size(0)) + " rows, " + std::to_string(l[0]) + " needed", ZC_ERR_CAPACITY);
        longest = t.size(0);
        return t.data_ptr();
    }

    // The given stream, or the current one; a stream that names a GPU (torch's
    // do) has to be the tensors' GPU's.
    hipStream_t stream(PyObject* o) {
        if (device >= 0 && device != c10::hip::current_device()) refuse("stream", "the tensors are not on the current GPU");
        if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
        if (PyObject* d = PyObject_GetAttrString(o, "device_index")) {
            const long index = PyLong_AsLong(d);
            Py_DECREF(d);
            if (index == -1 && PyErr_Occurred()) throw PythonError{};
            if (device >= 0 && index != device) refuse("stream", "not of the tensors' GPU");
        } else {
            PyErr_Clear();
        }
        PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
        if (!h) throw PythonError{};
        void* s = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!s && PyErr_Occurred()) throw PythonError{};
        return static_cast<hipStream_t>(s);
    }

private:
    int device = -1;
};

PyObject* const* items(PyObject* o, const char* what, Py_ssize_t n) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != n) refuse(what, "a tuple of " + std::to_string(n) + " expected");
    return &PyTuple_GET_ITEM(o, 0);
}

uint64_t number(PyObject* o, const char* what) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(what, "a number of 0 or more expected");
    }
    return v;
}

// What an ExpertPlan passes: (tokens, topk, experts, align, rows, workspace bytes).
struct Sizes {
    uint64_t tokens, rows, ws_bytes;
    uint32_t topk, experts, align;
    explicit Sizes(PyObject* o) {
        PyObject* const* v = items(o, "plan", 6);
        tokens = number(v[0], "tokens");
        topk = size32(number(v[1], "topk"), "topk");
        experts = size32(number(v[2], "experts"), "experts");
        align = size32(number(v[3], "align"), "align");
        rows = number(v[4], "rows");
        ws_bytes = number(v[5], "workspace");
    }
    uint64_t slots() const { return tokens * topk; }
};

// A routing as the calls read it; packed segments have no padding rows, which
// the library is told by counts 0.
struct Routing {
    const int32_t *offsets = nullptr, *counts = nullptr, *row;
    Routing(Call& c, const Sizes& s, PyObject* o) {
        PyObject* const* v = items(o, "routing", 4);
        row = c.flat<int32_t>(v[2], "row", at::kInt, s.slots());
        if (s.align == 1) return;
        offsets = c.flat<int32_t>(v[0], "offsets", at::kInt, s.experts + 1);
        counts = c.flat<int32_t>(v[1], "counts", at::kInt, s.experts);
    }
};

struct Blocks {
    void *data, *scale;
    uint64_t data_rows, scale_rows;
    Blocks(Call& c, PyObject* o, const char* what, uint64_t cols, std::initializer_list<uint64_t> lead,
           std::initializer_list<uint64_t> scale_lead) {
        PyObject* const* v = items(o, what, 3);
        const uint64_t have = number(v[2], what);
        if (have != cols) refuse(what, std::to_string(have) + " columns, " + std::to_string(cols) + " expected");
        data = c.part(v[0], what, at::kFloat8_e4m3fn, lead, up(cols, 128));
        data_rows = c.longest;
        scale = c.part(v[1], what, at::kFloat8_e8m0fnu, scale_lead, up((cols + 127) / 128, 4));
        scale_rows = c.longest;
    }
};

struct Columns {
    void *data, *scale;
    Columns(Call& c, PyObject* o, const char* what, uint64_t rows, uint64_t cols) {
        PyObject* const* v = items(o, what, 4);
        const uint64_t r = number(v[2], what), n = number(v[3], what);
        if (r != rows || n != cols)
            refuse(what, "columns of (" + std::to_string(r) + ", " + std::to_string(n) + "), (" + std::to_string(rows) +
                             ", " + std::to_string(cols) + ") expected");
        const uint64_t blocks = (rows + 127) / 128;
        data = c.part(v[0], what, at::kFloat8_e4m3fn, {blocks, cols}, 128);
        scale = c.part(v[1], what, at::kFloat8_e8m0fnu, {blocks}, up(cols, 4));
    }
};

// A 3-dimensional contiguous tensor of one of the three row types.
const at::Tensor& stack(Call& c, PyObject* o, const char* what) {
    const at::Tensor& t = c.tensor(o, what);
    if (t.dim() != 3 || dtype_of(t.scalar_type()) < 0)
        refuse(what, "shape " + shape_text(t.sizes()) + ", type " + c10::toString(t.scalar_type()));
    if (!t.is_contiguous()) refuse(what, "not contiguous");
    return t;
}

// The library's call, with other Python threads running: it may wait for room
// in a full queue.
template <typename F, typename... A>
void enqueue(const char* name, F f, A... args) {
    zc_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = f(args...);
    Py_END_ALLOW_THREADS;
    if (rc) throw Refused{rc, name};
}

typedef PyObject* const* Args;

void route(Args a) {  // sizes, ids, routing, ws, stream
    Call c;
    const Sizes z(a[0]);
    const int32_t* ids = c.flat<int32_t>(a[1], "ids", at::kInt, z.slots());
    PyObject* const* r = items(a[2], "routing", 4);
    int32_t* offsets = c.flat<int32_t>(r[0], "offsets", at::kInt, z.experts + 1);
    int32_t* counts = c.flat<int32_t>(r[1], "counts", at::kInt, z.experts);
    int32_t* row = c.flat<int32_t>(r[2], "row", at::kInt, z.slots());
    uint64_t slots = 0, bytes = 0;
    int32_t* slot = c.flat<int32_t>(r[3], "slot", at::kInt, z.rows, &slots);
    void* ws = c.flat(a[3], "workspace", at::kByte, z.ws_bytes, &bytes);
    enqueue("zc_route", zc.route, ids, z.tokens, z.topk, z.experts, z.align, offsets, counts, row, slot, slots, ws, bytes,
            c.stream(a[4]));
}

void dispatch(Args a) {  // sizes, x, routing, rows, stream
    Call c;
    const Sizes z(a[0]);
    const Matrix x = c.matrix(a[1], "x", z.tokens), rows = c.matrix(a[3], "rows", z.rows, x.dtype, x.width);
    const Routing r(c, z, a[2]);
    enqueue("zc_dispatch", zc.dispatch, x.p, x.stride, (uint32_t)x.dtype, z.tokens, z.topk, z.experts, x.width,
            r.offsets, r.counts, r.row, rows.p, rows.stride, rows.rows, c.stream(a[4]));
}

void dispatch_fp8(Args a) {  // sizes, x, routing, out, stream
    Call c;
    const Sizes z(a[0]);
    const Matrix x = c.matrix(a[1], "x", z.tokens);
    const Blocks out(c, a[3], "out", x.width, {z.rows}, {z.rows});
    const Routing r(c, z, a[2]);
    enqueue("zc_dispatch_fp8", zc.dispatch_fp8, x.p, x.stride, (uint32_t)x.dtype, z.tokens, z.topk, z.experts,
            x.width, r.offsets, r.counts, r.row, out.data, out.scale, std::min(out.data_rows, out.scale_rows),
            c.stream(a[4]));
}

void combine(Args a) {  // sizes, rows, weights, routing, y, stream
    Call c;
    const Sizes z(a[0]);
    const Matrix y = c.matrix(a[4], "y", z.tokens), rows = c.matrix(a[1], "rows", z.rows, y.dtype, y.width);
    const int32_t* row = c.flat<int32_t>(items(a[3], "routing", 4)[2], "row", at::kInt, z.slots());
    const float* w = c.flat_or_null<float>(a[2], "weights", at::kFloat, z.slots());
    enqueue("zc_combine", zc.combine, rows.p, rows.stride, w, (uint32_t)y.dtype, z.tokens, z.topk, y.width, row,
            rows.rows, y.p, y.stride, c.stream(a[5]));
}

void combine_backward(Args a) {  // sizes, dy, rows, weights, routing, drows, dweights, stream
    Call c;
    const Sizes z(a[0]);
    const Matrix dy = c.matrix(a[1], "dy", z.tokens);
    const Routing r(c, z, a[4]);
    if (a[5] == Py_None && a[6] == Py_None) refuse("combine_backward", "no gradient asked for");
    Matrix drows{nullptr, 0, 1ull << 31, 0, 0}, rows = drows;
    if (a[5] != Py_None) drows = c.matrix(a[5], "drows", z.rows, dy.dtype, dy.width);
    if (a[6] != Py_None) {
        if (a[2] == Py_None) refuse("combine_backward", "dweights needs rows");
        rows = c.matrix(a[2], "rows", z.rows, dy.dtype, dy.width);
    }
    const float* w = c.flat_or_null<float>(a[3], "weights", at::kFloat, z.slots());
    float* dw = c.flat_or_null<float>(a[6], "dweights", at::kFloat, z.slots());
    enqueue("zc_combine_backward", zc.combine_backward, dy.p, dy.stride, rows.p, rows.stride, w, (uint32_t)dy.dtype, z.tokens,
            z.topk, z.experts, dy.width, r.offsets, r.counts, r.row, std::min(drows.rows, rows.rows), drows.p,
            drows.stride, dw, c.stream(a[7]));
}

void quantize_rows(Args a) {  // x, out, used, stream
    Call c;
    const Matrix x = c.matrix(a[0], "x", 0);
    const Blocks out(c, a[1], "out", x.width, {x.rows}, {x.rows});
    const int32_t* used = c.flat_or_null<int32_t>(a[2], "used", at::kInt, 1);
    enqueue("zc_quantize_rows", zc.quantize_rows, x.p, x.stride, (uint32_t)x.dtype, x.rows, x.width, used, out.data,
            out.scale, c.stream(a[3]));
}

void quantize_weights(Args a) {  // w, out, transpose, stream
    Call c;
    const at::Tensor& w = stack(c, a[0], "w");
    const int transpose = PyObject_IsTrue(a[2]);
    if (transpose < 0) throw PythonError{};
    const uint32_t e = size32(w.size(0), "w"), n = size32(w.size(transpose ? 2 : 1), "w");
    const uint32_t k = size32(w.size(transpose ? 1 : 2), "w");
    const Blocks out(c, a[1], "out", k, {e, n}, {e, (n + 127ull) / 128});
    enqueue("zc_quantize_weights", zc.quantize_weights, w.data_ptr(), (uint32_t)dtype_of(w.scalar_type()), e, n, k, transpose, out.data, out.scale, c.stream(a[3]));
}

void quantize_columns(Args a) {  // x, out, used, stream
    Call c;
    const Matrix x = c.matrix(a[0], "x", 0);
    const Columns out(c, a[1], "out", x.rows, x.width);
    const int32_t* used = c.flat_or_null<int32_t>(a[2], "used", at::kInt, 1);
    enqueue("zc_quantize_columns", zc.quantize_columns, x.p, x.stride, (uint32_t)x.dtype, x.rows, x.width, used,
            out.data, out.scale, c.stream(a[3]));
}

void expert_product(Args a) {  // a, w, out, offsets, counts, stream
    Call c;
    PyObject* const* wt = items(a[1], "w", 3);
    const at::Tensor& w = c.tensor(wt[0], "w");
    if (w.dim() != 3) refuse("expert_product", "a is [rows, k], w is [experts, n, k]");
    const uint32_t experts = size32(w.size(0), "w"), n = size32(w.size(1), "w"), k = size32(number(wt[2], "w"), "w");
    const Matrix out = c.matrix(a[2], "out", 0, -1, n);
    const Blocks ab(c, a[0], "a", k, {out.rows}, {out.rows}), wb(c, a[1], "w", k, {experts, n},
        {experts, (n + 127ull) / 128});
    const int32_t* offsets = c.flat_or_null<int32_t>(a[3], "offsets", at::kInt, experts + 1ull);
    const int32_t* counts = c.flat_or_null<int32_t>(a[4], "counts", at::kInt, experts);
    enqueue("zc_expert_product", zc.expert_product, ab.data, ab.scale, out.rows, wb.data, wb.scale, experts,
            n, k, offsets, counts, out.p, out.stride, (uint32_t)out.dtype, c.stream(a[5]));
}

void expert_weight_grad(Args a) {  // y, x, dw, offsets, ws, stream
    Call c;
    const at::Tensor& dw = stack(c, a[2], "dw");
    const uint32_t experts = size32(dw.size(0), "dw"), n = size32(dw.size(1), "dw"), k = size32(dw.size(2), "dw");
    const uint64_t rows = number(items(a[1], "x", 4)[2], "x");
    const Columns y(c, a[0], "y", rows, n), x(c, a[1], "x", rows, k);
    const int32_t* offsets = c.flat_or_null<int32_t>(a[3], "offsets", at::kInt, (uint64_t)experts + 1);
    const uint64_t need = zc.expert_weight_grad_workspace_bytes(rows, experts, n, k);
    at::Tensor own;  // from torch's allocator, on the current stream, which is the call's
    void* ws = nullptr;
    if (need && a[4] != Py_None) ws = c.flat(a[4], "workspace", at::kByte, need);
    else if (need) ws = (own = at::empty({(int64_t)need}, dw.options().dtype(at::kByte))).data_ptr();
    enqueue("zc_expert_weight_grad", zc.expert_weight_grad, y.data, y.scale, x.data, x.scale, rows, experts, n, k, offsets,
            dw.data_ptr(), (uint32_t)dtype_of(dw.scalar_type()), ws, need, c.stream(a[5]));
}

// A call as Python makes it: exactly N positional arguments, every C++
// exception turned into Python's.
template <void (*F)(Args), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    try {
        if (n != N) throw Refused{ZC_ERR_INVALID_ARG, "number of arguments"};
        F(args);
        Py_RETURN_NONE;
    } catch (const Refused& r) {
        if (!error_type) {
            PyErr_SetString(PyExc_RuntimeError, r.what.c_str());
        } else if (PyObject* e = PyObject_CallFunction(error_type, "is", r.code, r.what.c_str())) {
            PyErr_SetObject(error_type, e);
            Py_DECREF(e);
        }
    } catch (const PythonError&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(error type, {symbol: address})
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 2 || !PyDict_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "bind(error type, {symbol: address})");
        return nullptr;
    }
    auto get = [&](const char* name, auto& f) {
        PyObject* v = PyDict_GetItemString(args[1], name);
        void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
        if (p) f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(p);
        else if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, name);
        return p != nullptr;
    };
    const bool all = get("zc_route", zc.route) && get("zc_dispatch", zc.dispatch) &&
                     get("zc_dispatch_fp8", zc.dispatch_fp8) && get("zc_combine", zc.combine) &&
                     get("zc_combine_backward", zc.combine_backward) && get("zc_quantize_rows", zc.quantize_rows) &&
                     get("zc_quantize_weights", zc.quantize_weights) && get("zc_quantize_columns", zc.quantize_columns) &&
                     get("zc_expert_product", zc.expert_product) && get("zc_expert_weight_grad", zc.expert_weight_grad) &&
                     get("zc_expert_weight_grad_workspace_bytes", zc.expert_weight_grad_workspace_bytes);
    if (!all) return nullptr;
    Py_INCREF(args[0]);
    Py_XDECREF(error_type);
    error_type = args[0];
    Py_RETURN_NONE;
}

#define CALL(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    CALL(route, 5), CALL(dispatch, 5), CALL(dispatch_fp8, 5), CALL(combine, 6), CALL(combine_backward, 8),
    CALL(quantize_rows, 4), CALL(quantize_weights, 4), CALL(quantize_columns, 4), CALL(expert_product, 6),
    CALL(expert_weight_grad, 6), {nullptr, nullptr, 0, nullptr}};
#undef CALL

PyModuleDef module = {PyModuleDef_HEAD_INIT, "zc_experts_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_zc_experts_binding() { return PyModule_Create(&module); }
