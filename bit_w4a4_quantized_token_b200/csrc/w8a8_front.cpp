// w8a8_front.cpp -- the host side of a W8A8 layer call, as a CPython module:
// checks of the torch operands (what the C ABI cannot see behind a pointer),
// allocation of the outputs, and the call of the library's entry point on the
// operands' GPU and its current stream.  No arithmetic of the layer.
//
// A call on few tokens is bound by what the host does for it.  The same work
// in Python took, per call, 6.4 us (quantise), 9.1 (norm) and 7.2 (GEMM), of
// which the library's own part is 2.2 to 2.9: against 8 us of GPU time for a
// one-token linear of 4096 x 4096, the host was twice as slow as the GPU.
//
// The entry points' addresses come from the ctypes binding (bind), so that
// the library is loaded once, by the binding, wherever that found it.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "svdq.h"

namespace {

using at::Tensor;

decltype(&svdq_pack_weight_w8a8) g_pack = nullptr;
decltype(&svdq_quantize_act_w8a8) g_quantize = nullptr;
decltype(&svdq_rms_norm_quantize_w8a8) g_norm = nullptr;
decltype(&svdq_gemm_w8a8) g_gemm = nullptr;
PyObject* g_raise = nullptr;   // raise_status(status, entry point's name): raises the binding's error

// A refusal: becomes a ValueError at the module's boundary.
struct Refused {
    std::string text;
};

std::string describe(const Tensor& t) {
    return c10::str(t.dtype(), " ", t.sizes(), " (strides ", t.strides(), ") on ", t.device());
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw Refused{c10::str(name, ": expected a tensor")};
    return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

int64_t whole(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused{c10::str(name, ": expected a whole number")};
    }
    return v;
}

// The library's type, or -1.
int type_of(const Tensor& t) {
    const auto s = t.scalar_type();
    return s == at::kBFloat16 ? SVDQ_BF16 : s == at::kHalf ? SVDQ_F16 : s == at::kFloat ? SVDQ_F32 : -1;
}
at::ScalarType scalar_of(int type) {
    return type == SVDQ_BF16 ? at::kBFloat16 : type == SVDQ_F16 ? at::kHalf : at::kFloat;
}

bool has_shape(const Tensor& t, int64_t rows, int64_t cols) {   // cols < 0: a vector
    return cols < 0 ? t.dim() == 1 && t.size(0) == rows : t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

// A contiguous operand; returns its address.
void* fixed(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t cols, int64_t index) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != type || !has_shape(t, rows, cols) || t.get_device() != index || !t.is_contiguous())
        throw Refused{c10::str(name, ": expected a contiguous ", type, " tensor of shape [", rows,
                               cols < 0 ? std::string() : c10::str(", ", cols), "] on GPU ", index, ", got ",
                               describe(t))};
    return t.data_ptr();
}
void* fixed_or_null(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t cols, int64_t index) {
    return given(o) ? fixed(o, name, type, rows, cols, index) : nullptr;
}

// A matrix of activations: rows may be apart, elements of a row not.
struct Rows {
    const Tensor& t;
    int type;
    int64_t M, ld;
};
Rows rows_of(PyObject* o, const char* name, int64_t K) {
    const Tensor& t = tensor(o, name);
    const int type = type_of(t);
    if (type < 0 || t.dim() != 2 || t.size(1) != K || t.stride(1) != 1 || !t.is_cuda())
        throw Refused{c10::str(name, ": expected a CUDA matrix [M, ", K,
                               "] of bf16, fp16 or fp32 with contiguous rows, got ", describe(t))};
    return {t, type, t.size(0), t.size(0) > 1 ? t.stride(0) : K};
}

Tensor empty(at::ScalarType type, std::initializer_list<int64_t> shape, int64_t index) {
    return Tensor(at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), type,
                                         at::Device(at::kCUDA, (c10::DeviceIndex)index), c10::nullopt));
}

svdq_stream_t stream_of(int64_t index) {
    return reinterpret_cast<svdq_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream());
}

// An output: the caller's, or a new tensor.
PyObject* keep_or_wrap(PyObject* o, Tensor&& made) {
    if (given(o)) {
        Py_INCREF(o);
        return o;
    }
    return THPVariable_Wrap(std::move(made));
}

PyObject* fail(svdq_status status, const char* name) {
    PyObject* r = PyObject_CallFunction(g_raise, "is", (int)status, name);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: status %d", name, (int)status);
    return nullptr;
}

#define W8_BEGIN(count)                                                                           \
    HANDLE_TH_ERRORS                                                                              \
    if (n != (count)) return PyErr_Format(PyExc_TypeError, "expected %d arguments", (int)(count)); \
    try {
#define W8_END                                             \
    }                                                      \
    catch (const Refused& r) {                             \
        PyErr_SetString(PyExc_ValueError, r.text.c_str()); \
        return nullptr;                                    \
    }                                                      \
    END_HANDLE_TH_ERRORS

// pack(W, lam or None) -> (codes, scales, inv_lambda or None)
PyObject* pack(PyObject*, PyObject* const* a, Py_ssize_t n) {
    W8_BEGIN(2)
    const Tensor& given_w = tensor(a[0], "W");
    const Rows w0 = rows_of(a[0], "W", given_w.dim() == 2 ? given_w.size(1) : -1);
    const int64_t N = w0.M, K = given_w.size(1), index = given_w.get_device();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    void* lam = fixed_or_null(a[1], "lam", at::kFloat, K, -1, index);
    const Tensor w = given_w.contiguous();
    Tensor codes = empty(at::kChar, {N, K}, index), scales = empty(at::kFloat, {N}, index), inv;
    if (lam) inv = empty(at::kFloat, {K}, index);
    const svdq_status st = g_pack((svdq_dtype)w0.type, w.data_ptr(), N, K, (const float*)lam, codes.data_ptr(),
                                  (float*)scales.data_ptr(), lam ? (float*)inv.data_ptr() : nullptr, stream_of(index));
    if (st != SVDQ_OK) return fail(st, "svdq_pack_weight_w8a8");
    PyObject* i = Py_None;
    if (lam)
        i = THPVariable_Wrap(std::move(inv));
    else
        Py_INCREF(i);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(codes)), THPVariable_Wrap(std::move(scales)), i);
    W8_END
}

// quantize(x, K, inv_lambda or None, codes or None, scales or None) -> (M, codes, scales)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
    W8_BEGIN(5)
    const int64_t K = whole(a[1], "K");
    const Rows x = rows_of(a[0], "x", K);
    const int64_t index = x.t.get_device();
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    void* inv = fixed_or_null(a[2], "packed.inv_lambda", at::kFloat, K, -1, index);
    void* codes = fixed_or_null(a[3], "out.x_codes", at::kChar, x.M, K, index);
    void* scales = fixed_or_null(a[4], "out.x_scales", at::kFloat, x.M, -1, index);
    Tensor new_codes, new_scales;
    if (!codes) codes = (new_codes = empty(at::kChar, {x.M, K}, index)).data_ptr();
    if (!scales) scales = (new_scales = empty(at::kFloat, {x.M}, index)).data_ptr();
    const svdq_status st = g_quantize((svdq_dtype)x.type, x.t.data_ptr(), x.ld, x.M, K, (const float*)inv, codes,
                                      (float*)scales, stream_of(index));
    if (st != SVDQ_OK) return fail(st, "svdq_quantize_act_w8a8");
    return Py_BuildValue("(LNN)", (long long)x.M, keep_or_wrap(a[3], std::move(new_codes)),
                         keep_or_wrap(a[4], std::move(new_scales)));
    W8_END
}

// norm(x, residual, norm_weight, K, inv_lambda, eps, h_out, normed, codes, scales) -> (h, M, codes, scales);
// all but x, K and eps may be None
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    W8_BEGIN(10)
    const int64_t K = whole(a[3], "K");
    const Rows x = rows_of(a[0], "x", K);
    const int64_t index = x.t.get_device();
    const auto type = scalar_of(x.type);
    const double eps = PyFloat_AsDouble(a[5]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    void* residual = nullptr;
    int64_t ldr = K;
    if (given(a[1])) {
        const Rows r = rows_of(a[1], "residual", K);
        if (r.type != x.type || r.M != x.M || r.t.get_device() != index)
            throw Refused{c10::str("residual: expected what x is, ", describe(x.t), ", got ", describe(r.t))};
        residual = r.t.data_ptr();
        ldr = r.ld;
    }
    void* weight = fixed_or_null(a[2], "norm_weight", type, K, -1, index);
    void* inv = fixed_or_null(a[4], "packed.inv_lambda", at::kFloat, K, -1, index);
    void* h = fixed_or_null(a[6], "h_out", type, x.M, K, index);
    void* normed = fixed_or_null(a[7], "normed", type, x.M, K, index);
    void* codes = fixed_or_null(a[8], "out.x_codes", at::kChar, x.M, K, index);
    void* scales = fixed_or_null(a[9], "out.x_scales", at::kFloat, x.M, -1, index);
    Tensor new_h, new_codes, new_scales;
    if (!h && residual) h = (new_h = empty(type, {x.M, K}, index)).data_ptr();
    if (!codes) codes = (new_codes = empty(at::kChar, {x.M, K}, index)).data_ptr();
    if (!scales) scales = (new_scales = empty(at::kFloat, {x.M}, index)).data_ptr();
    const svdq_status st =
        g_norm((svdq_dtype)x.type, x.t.data_ptr(), x.ld, residual, ldr, x.M, K, weight, (float)eps, (const float*)inv, h,
               normed, codes, (float*)scales, stream_of(index));
    if (st != SVDQ_OK) return fail(st, "svdq_rms_norm_quantize_w8a8");
    // without a residual and an h_out, h is x itself
    return Py_BuildValue("(NLNN)", keep_or_wrap(!given(a[6]) && !residual ? a[0] : a[6], std::move(new_h)),
                         (long long)x.M, keep_or_wrap(a[8], std::move(new_codes)),
                         keep_or_wrap(a[9], std::move(new_scales)));
    W8_END
}

// gemm(x_codes, x_scales, M, w_codes, w_scales, N, K, bias or None, y_type, y or None) -> y
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    W8_BEGIN(10)
    const int64_t M = whole(a[2], "M"), N = whole(a[5], "N"), K = whole(a[6], "K");
    const int y_type = (int)whole(a[8], "y_type");
    const auto type = scalar_of(y_type);
    const int64_t index = tensor(a[0], "q.x_codes").get_device();
    void* x_codes = fixed(a[0], "q.x_codes", at::kChar, M, K, index);
    void* x_scales = fixed(a[1], "q.x_scales", at::kFloat, M, -1, index);
    void* w_codes = fixed(a[3], "packed.w_codes", at::kChar, N, K, index);
    void* w_scales = fixed(a[4], "packed.w_scales", at::kFloat, N, -1, index);
    void* bias = fixed_or_null(a[7], "packed.bias", type, N, -1, index);
    void* y = fixed_or_null(a[9], "y", type, M, N, index);
    if (index < 0) throw Refused{"q.x_codes: expected CUDA tensors, got tensors on the CPU"};
    const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
    Tensor new_y;
    if (!y) y = (new_y = empty(type, {M, N}, index)).data_ptr();
    const svdq_status st = g_gemm(x_codes, (const float*)x_scales, M, w_codes, (const float*)w_scales, N, K, bias,
                                  (svdq_dtype)y_type, y, stream_of(index));
    if (st != SVDQ_OK) return fail(st, "svdq_gemm_w8a8");
    return keep_or_wrap(a[9], std::move(new_y));
    W8_END
}

// bind(pack, quantize, norm, gemm addresses, raise_status)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    W8_BEGIN(5)
    g_pack = reinterpret_cast<decltype(g_pack)>((uintptr_t)whole(a[0], "pack"));
    g_quantize = reinterpret_cast<decltype(g_quantize)>((uintptr_t)whole(a[1], "quantize"));
    g_norm = reinterpret_cast<decltype(g_norm)>((uintptr_t)whole(a[2], "norm"));
    g_gemm = reinterpret_cast<decltype(g_gemm)>((uintptr_t)whole(a[3], "gemm"));
    Py_INCREF(a[4]);
    Py_XDECREF(g_raise);
    g_raise = a[4];
    Py_RETURN_NONE;
    W8_END
}

#define W8_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {W8_METHOD(bind), W8_METHOD(pack), W8_METHOD(quantize), W8_METHOD(norm), W8_METHOD(gemm),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w8a8_front", "Host side of a W8A8 layer call.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w8a8_front() { return PyModule_Create(&module); }
