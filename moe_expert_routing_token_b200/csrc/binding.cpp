// Python binding of the expert layer's calls (module _experts): checks of the
// tensors, allocation of the outputs, and the C entry points of
// include/moe_routing.h on the operands' device and its current stream.
//
// These calls are small next to their checks: at decode sizes a kernel takes
// 3 us, the same checks and the call through ctypes took 9 to 10.
// experts.py documents the functions and gives them their arguments by
// position.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "moe_routing.h"

namespace {

using at::Tensor;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kI32 = at::kInt;

std::string shape_text(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, " is out of range");
    return v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

// Sizes as the C entry points take them.
int32_t i32(int64_t v, const char* name) {
    TORCH_CHECK_VALUE(v <= INT32_MAX, name, " = ", v, " is out of range");
    return (int32_t)v;
}

void rows(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.dim() == 2 && t.is_contiguous(), name, " must be a contiguous 2-D tensor");
}

void expect(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& beside) {
    TORCH_CHECK_VALUE(t.sizes() == shape && t.scalar_type() == dtype && t.is_contiguous() &&
                          t.device() == beside.device(),
                      name, " must be a contiguous ", shape_text(shape), " ", dtype, " tensor on ", beside.device());
}

// The tensor given for an output, or none.
const Tensor* given(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

// That tensor, checked, or a new one on the device of `beside`.
Tensor output(const Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& beside) {
    if (t != nullptr) {
        expect(*t, name, shape, dtype, beside);
        return *t;
    }
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(beside.device()));
}

int dtype_code(const Tensor& t) {
    TORCH_CHECK_VALUE(t.scalar_type() == kF32 || t.scalar_type() == kBf16, "unsupported dtype ", t.scalar_type(),
                      "; expected float32 or bfloat16");
    return t.scalar_type() == kF32 ? MOE_DTYPE_F32 : MOE_DTYPE_BF16;
}

void places(const Tensor& scatter, int64_t pairs, const Tensor& beside) {
    TORCH_CHECK_VALUE(scatter.scalar_type() == kI32 && scatter.numel() == pairs && scatter.is_contiguous() &&
                          scatter.device() == beside.device(),
                      "scatter_indx must be a contiguous int32 tensor of ", pairs, " places on ", beside.device());
}

void on_gpu(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
}

// Around allocations and launches: makes the operands' device current, knows
// its stream, and lets other Python threads run, as either may wait for the
// device.
struct Launch {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream;
    PyThreadState* state;
    explicit Launch(const Tensor& t) {
        const auto index = t.device().index();
        if (c10::cuda::current_device() != index) guard.set_index(index);
        stream = c10::cuda::getCurrentCUDAStream(index).stream();
        state = PyEval_SaveThread();
    }
    Launch(const Launch&) = delete;
    ~Launch() { lock(); }
    void lock() {
        if (state != nullptr) PyEval_RestoreThread(state);
        state = nullptr;
    }
};

void check(Launch& l, int status, const char* name) {
    l.lock();
    if (status == MOE_OK) return;
    const std::string text = std::string(name) + ": " + moe_last_error();
    PyObject* kind = status == MOE_ERR_INVALID_ARG ? PyExc_ValueError
                     : status == MOE_ERR_UNSUPPORTED ? PyExc_NotImplementedError : PyExc_RuntimeError;
    if (status == MOE_ERR_CUDA) {
        if (PyObject* m = PyImport_ImportModule("moe_expert_routing_token_b200.routing")) {
            if (PyObject* c = PyObject_GetAttrString(m, "RoutingError")) kind = c;  // kept alive by its module
            Py_DECREF(m);
        }
        PyErr_Clear();
    }
    PyErr_SetString(kind, text.c_str());
    throw python_error();
}

PyObject* two(const Tensor& a, const Tensor& b) {
    PyObject* t = PyTuple_New(2);
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
    TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

const void* data(PyObject* o, const Tensor& t) { return o == Py_None ? nullptr : t.const_data_ptr(); }

// (x, scatter_indx, topk, out)
PyObject* gather_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 4);
    const Tensor &x = tensor(a[0], "x"), &scatter = tensor(a[1], "scatter_indx");
    const int64_t k = integer(a[2], "topk");
    rows(x, "x");
    const int code = dtype_code(x);
    TORCH_CHECK_VALUE(k >= 1, "topk must be positive");
    const int64_t M = x.size(0), H = x.size(1);
    places(scatter, M * k, x);
    on_gpu(x, "x");
    const Tensor* to = given(a[3], "out");
    Launch l(x);
    Tensor out = output(to, "out", {M * k, H}, x.scalar_type(), x);
    check(l, moe_gather_tokens(x.const_data_ptr(), code, M, i32(H, "H"), (const int32_t*)scatter.const_data_ptr(),
                               (int)k, out.mutable_data_ptr(), l.stream),
          "moe_gather_tokens");
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (grad_sorted, scatter_indx, topk, out)
PyObject* gather_tokens_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 4);
    const Tensor &g = tensor(a[0], "grad_sorted"), &scatter = tensor(a[1], "scatter_indx");
    const int64_t k = integer(a[2], "topk");
    rows(g, "grad_sorted");
    const int code = dtype_code(g);
    TORCH_CHECK_VALUE(k >= 1 && g.size(0) % k == 0, "grad_sorted must have a row for each of the tokens' ", k,
                      " slots");
    const int64_t M = g.size(0) / k, H = g.size(1);
    places(scatter, M * k, g);
    on_gpu(g, "grad_sorted");
    const Tensor* to = given(a[3], "out");
    Launch l(g);
    Tensor out = output(to, "out", {M, H}, g.scalar_type(), g);
    check(l, moe_gather_tokens_backward(g.const_data_ptr(), code, M, i32(H, "H"),
                                        (const int32_t*)scatter.const_data_ptr(), (int)k, out.mutable_data_ptr(),
                                        l.stream),
          "moe_gather_tokens_backward");
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (y, scatter_indx, topk_weights, residual, out)
PyObject* combine_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 5);
    const Tensor &y = tensor(a[0], "y"), &scatter = tensor(a[1], "scatter_indx"), &w = tensor(a[2], "topk_weights");
    rows(y, "y");
    rows(w, "topk_weights");
    const int code = dtype_code(y);
    const int64_t M = w.size(0), k = w.size(1), H = y.size(1);
    expect(w, "topk_weights", {M, k}, kF32, y);
    TORCH_CHECK_VALUE(y.size(0) == M * k, "y must have a row for each of the ", M * k, " places");
    places(scatter, M * k, y);
    const Tensor& r = a[3] == Py_None ? y : tensor(a[3], "residual");
    if (a[3] != Py_None) expect(r, "residual", {M, H}, y.scalar_type(), y);
    on_gpu(y, "y");
    const Tensor* to = given(a[4], "out");
    Launch l(y);
    Tensor out = output(to, "out", {M, H}, y.scalar_type(), y);
    check(l, moe_combine_tokens(y.const_data_ptr(), code, M, i32(H, "H"), (const int32_t*)scatter.const_data_ptr(),
                                i32(k, "topk"), (const float*)w.const_data_ptr(), data(a[3], r),
                                out.mutable_data_ptr(), l.stream),
          "moe_combine_tokens");
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (grad_out, y, scatter_indx, topk_weights, grad_y, grad_weights)
PyObject* combine_tokens_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const Tensor &g = tensor(a[0], "grad_out"), &y = tensor(a[1], "y"), &scatter = tensor(a[2], "scatter_indx"),
                 &w = tensor(a[3], "topk_weights");
    rows(g, "grad_out");
    rows(w, "topk_weights");
    const int code = dtype_code(g);
    const int64_t M = w.size(0), k = w.size(1), H = g.size(1);
    expect(w, "topk_weights", {M, k}, kF32, g);
    TORCH_CHECK_VALUE(g.size(0) == M, "grad_out must have a row for each of the ", M, " tokens");
    expect(y, "y", {M * k, H}, g.scalar_type(), g);
    places(scatter, M * k, g);
    on_gpu(g, "grad_out");
    const Tensor *to_y = given(a[4], "grad_y"), *to_w = given(a[5], "grad_weights");
    Launch l(g);
    Tensor gy = output(to_y, "grad_y", {M * k, H}, g.scalar_type(), g);
    Tensor gw = output(to_w, "grad_weights", {M, k}, kF32, g);
    check(l, moe_combine_tokens_backward(g.const_data_ptr(), y.const_data_ptr(), code, M, i32(H, "H"),
                                         (const int32_t*)scatter.const_data_ptr(), i32(k, "topk"),
                                         (const float*)w.const_data_ptr(), gy.mutable_data_ptr(),
                                         (float*)gw.mutable_data_ptr(), l.stream),
          "moe_combine_tokens_backward");
    return two(gy, gw);
    END_HANDLE_TH_ERRORS
}

// Checks of a sorted row array and the offsets; the number of experts.
int64_t experts(const Tensor& t, const char* name, const Tensor& offsets) {
    rows(t, name);
    TORCH_CHECK_VALUE(t.scalar_type() == kBf16, name, " must be bfloat16");
    TORCH_CHECK_VALUE(offsets.scalar_type() == kI32 && offsets.dim() == 1 && offsets.numel() >= 2 &&
                          offsets.is_contiguous() && offsets.device() == t.device(),
                      "expert_offsets must be a contiguous int32 tensor of E + 1 values on ", t.device());
    return offsets.numel() - 1;
}

void expert_weight(const Tensor& w, int64_t E, const Tensor& beside) {
    TORCH_CHECK_VALUE(w.scalar_type() == kBf16 && w.dim() == 3 && w.size(0) == E && w.is_contiguous() &&
                          w.device() == beside.device(),
                      "weight must be a contiguous bfloat16 tensor (E = ", E, ", N, K) on ", beside.device());
}

// (x, weight, expert_offsets, bias, activation, gated, residual, return_preact, out, preact_out)
PyObject* expert_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 10);
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "weight"), &offsets = tensor(a[2], "expert_offsets");
    const int64_t act = integer(a[4], "activation");
    const bool gated = truth(a[5]), kept = truth(a[7]) || a[9] != Py_None;
    const int64_t E = experts(x, "x", offsets);
    expert_weight(w, E, x);
    const int64_t P = x.size(0), K = x.size(1), Nz = w.size(1);
    TORCH_CHECK_VALUE(w.size(2) == K && !(gated && Nz % 2),
                      "weight does not match x's columns, or a gated weight has an odd number of rows");
    const int64_t N = gated ? Nz / 2 : Nz;
    const Tensor &bias = a[3] == Py_None ? x : tensor(a[3], "bias"),
                 &residual = a[6] == Py_None ? x : tensor(a[6], "residual");
    if (a[3] != Py_None) expect(bias, "bias", {E, Nz}, kF32, x);
    if (a[6] != Py_None) expect(residual, "residual", {P, N}, kBf16, x);
    on_gpu(x, "x");
    const Tensor *to = given(a[8], "out"), *to_preact = given(a[9], "preact_out");
    Launch l(x);
    Tensor out = output(to, "out", {P, N}, kBf16, x), preact;
    if (kept) preact = output(to_preact, "preact_out", {P, Nz}, kBf16, x);
    check(l, moe_expert_matmul(x.const_data_ptr(), w.const_data_ptr(), (const int32_t*)offsets.const_data_ptr(), P,
                               i32(K, "K"), i32(N, "N"), i32(E, "E"), (const float*)data(a[3], bias), (int)act,
                               gated, data(a[6], residual), out.mutable_data_ptr(),
                               kept ? preact.mutable_data_ptr() : nullptr, l.stream),
          "moe_expert_matmul");
    return kept ? two(out, preact) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (grad_out, weight, expert_offsets, preact, activation, gated, out)
PyObject* expert_matmul_grad_input(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 7);
    const Tensor &g = tensor(a[0], "grad_out"), &w = tensor(a[1], "weight"), &offsets = tensor(a[2], "expert_offsets");
    const int64_t act = integer(a[4], "activation");
    const bool gated = truth(a[5]);
    const int64_t E = experts(g, "grad_out", offsets);
    expert_weight(w, E, g);
    const int64_t P = g.size(0), N = g.size(1), K = w.size(2);
    TORCH_CHECK_VALUE(w.size(1) == N, "weight does not match grad_out's columns");
    const int64_t width = gated ? 2 * K : K;
    TORCH_CHECK_VALUE(a[3] != Py_None || (act == MOE_ACT_NONE && !gated), "an activation's gradient needs its preact");
    const Tensor& preact = a[3] == Py_None ? g : tensor(a[3], "preact");
    if (a[3] != Py_None) expect(preact, "preact", {P, width}, kBf16, g);
    on_gpu(g, "grad_out");
    const Tensor* to = given(a[6], "out");
    Launch l(g);
    Tensor out = output(to, "out", {P, width}, kBf16, g);
    check(l, moe_expert_matmul_grad_input(g.const_data_ptr(), w.const_data_ptr(),
                                          (const int32_t*)offsets.const_data_ptr(), P, i32(K, "K"), i32(N, "N"),
                                          i32(E, "E"), data(a[3], preact), (int)act, gated, out.mutable_data_ptr(),
                                          l.stream),
          "moe_expert_matmul_grad_input");
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (grad_out, x, expert_offsets, bias_grad, fp32, out)
PyObject* expert_matmul_grad_weight(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 6);
    const Tensor &g = tensor(a[0], "grad_out"), &x = tensor(a[1], "x"), &offsets = tensor(a[2], "expert_offsets");
    const bool bias = truth(a[3]);
    const int64_t E = experts(g, "grad_out", offsets);
    TORCH_CHECK_VALUE(x.dim() == 2, "x must be 2-D");
    const int64_t P = g.size(0), N = g.size(1), K = x.size(1);
    expect(x, "x", {P, K}, kBf16, g);
    auto dtype = truth(a[4]) ? kF32 : kBf16;
    const Tensor* to = given(a[5], "out");
    if (to != nullptr) dtype = to->scalar_type();
    TORCH_CHECK_VALUE(dtype == kF32 || dtype == kBf16, "unsupported dtype ", dtype, "; expected float32 or bfloat16");
    on_gpu(g, "grad_out");
    Launch l(g);
    Tensor out = output(to, "out", {E, N, K}, dtype, g), db;
    if (bias) db = output(nullptr, "grad_bias", {E, N}, kF32, g);
    check(l, moe_expert_matmul_grad_weight(g.const_data_ptr(), x.const_data_ptr(),
                                           (const int32_t*)offsets.const_data_ptr(), P, i32(K, "K"), i32(N, "N"),
                                           i32(E, "E"), dtype_code(out), out.mutable_data_ptr(),
                                           bias ? (float*)db.mutable_data_ptr() : nullptr, l.stream),
          "moe_expert_matmul_grad_weight");
    return bias ? two(out, db) : THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

// (grad_weights, gating_output, topk_ids, scoring, renormalize, routed_scaling_factor, softcap, out)
PyObject* topk_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arguments(n, 8);
    const Tensor &g = tensor(a[0], "grad_weights"), &x = tensor(a[1], "gating_output"), &ids = tensor(a[2], "topk_ids");
    const int64_t scoring = integer(a[3], "scoring");
    const bool renorm = truth(a[4]);
    const double rsf = number(a[5]), cap = number(a[6]);
    rows(x, "gating_output");
    const int code = dtype_code(x);
    TORCH_CHECK_VALUE(ids.dim() == 2, "topk_ids must be 2-D");
    const int64_t M = x.size(0), E = x.size(1), k = ids.size(1);
    expect(ids, "topk_ids", {M, k}, kI32, x);
    expect(g, "grad_weights", {M, k}, kF32, x);
    on_gpu(x, "gating_output");
    const Tensor* to = given(a[7], "out");
    Launch l(x);
    Tensor out = output(to, "out", {M, E}, x.scalar_type(), x);
    check(l, moe_topk_backward((const float*)g.const_data_ptr(), x.const_data_ptr(), code,
                               (const int32_t*)ids.const_data_ptr(), M, i32(E, "E"), i32(k, "topk"), (int)scoring,
                               renorm, (float)rsf, (float)cap, out.mutable_data_ptr(), l.stream),
          "moe_topk_backward");
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

#define MOE_METHOD(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {MOE_METHOD(gather_tokens),
                         MOE_METHOD(gather_tokens_backward),
                         MOE_METHOD(combine_tokens),
                         MOE_METHOD(combine_tokens_backward),
                         MOE_METHOD(expert_matmul),
                         MOE_METHOD(expert_matmul_grad_input),
                         MOE_METHOD(expert_matmul_grad_weight),
                         MOE_METHOD(topk_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__experts() { return PyModule_Create(&module); }
