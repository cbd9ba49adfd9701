// Argument marshalling of the operators between the adapted linears, for
// Python: checks the tensors, allocates a result that is not given, picks the
// stream and calls the C ABI, whose entry points the package hands over once
// (install).  No arithmetic.  A decode step makes these calls for one token at
// a time; through ctypes the checks and the conversion of the arguments took
// two to four times the launch itself (rotary 12.4 us, now 4-5).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <optional>

#include "adafuse.h"

namespace {

decltype(&adafuse_project) project_fn;
decltype(&adafuse_gated_project) gated_fn;
decltype(&adafuse_epilogue) epilogue_fn;
decltype(&adafuse_rotary) rotary_fn;

using at::Tensor;

// ValueError
template <typename... A>
[[noreturn]] void refuse(const A&... a)
{
    TORCH_CHECK_VALUE(false, a...);
    __builtin_unreachable();
}

const Tensor* optional_tensor(PyObject* o, const char* name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(name, " is not a tensor");
    return &THPVariable_Unpack(o);
}

const Tensor& tensor(PyObject* o, const char* name)
{
    const Tensor* t = optional_tensor(o, name);
    if (!t) refuse(name, " is missing");
    return *t;
}

const Tensor& matrix(PyObject* o, const char* name)
{
    const Tensor& t = tensor(o, name);
    if (t.dim() != 2) refuse(name, " has shape ", t.sizes(), "; expected two dimensions");
    return t;
}

// A [rows, n] operand whose rows' elements are adjacent; its row stride.
int64_t rows(const Tensor& t, const char* name, at::ScalarType type, int64_t r, int64_t n, at::Device dev)
{
    if (t.dim() != 2 || t.size(0) != r || t.size(1) != n || t.scalar_type() != type || t.device() != dev)
        refuse(name, " is ", t.scalar_type(), " ", t.sizes(), " on ", t.device(), "; expected ", type, " [", r, ", ", n,
               "] on ", dev);
    if (t.stride(1) != 1 && n > 1) refuse(name, ": the elements of a row must be adjacent (strides ", t.strides(), ")");
    return t.stride(0);
}

void* vector(const Tensor* t, const char* name, at::ScalarType type, int64_t n, at::Device dev)
{
    if (!t) return nullptr;
    if (t->dim() != 1 || t->size(0) != n || t->scalar_type() != type || t->device() != dev ||
        (t->stride(0) != 1 && n > 1))
        refuse(name, ": expected ", n, " adjacent elements of ", type, " on ", dev, ", got ", t->scalar_type(), " ",
               t->sizes(), " on ", t->device());
    return t->data_ptr();
}

// Makes the call's device and stream current for what the call allocates.
// `stream`: None for the device's current one, or the raw stream.
struct On {
    std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
    std::optional<c10::cuda::CUDAGuard> device_guard;
    cudaStream_t raw;
    On(at::Device dev, PyObject* stream)
    {
        if (!dev.is_cuda()) refuse("expected CUDA tensors, got ", dev);
        if (stream == Py_None) {
            if (dev.index() != c10::cuda::current_device()) device_guard.emplace(dev);
            raw = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
            return;
        }
        raw = reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(stream));
        if (PyErr_Occurred()) throw python_error();
        stream_guard.emplace(raw ? c10::cuda::getStreamFromExternal(raw, dev.index())
                                 : c10::cuda::getDefaultCUDAStream(dev.index()));
    }
};

at::ScalarType result_type(const Tensor* out, PyObject* dtype)
{
    std::optional<at::ScalarType> asked;
    if (dtype != Py_None) {
        if (!THPDtype_Check(dtype)) refuse("out_dtype is not a dtype");
        asked = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
    }
    const at::ScalarType t = out ? out->scalar_type() : asked.value_or(at::kBFloat16);
    if ((t != at::kBFloat16 && t != at::kFloat) || (asked && *asked != t)) refuse("the result is bfloat16 or float32");
    return t;
}

uint32_t flags_of(PyObject* o)
{
    const unsigned long v = PyLong_AsUnsignedLong(o);
    if (PyErr_Occurred()) throw python_error();
    return (uint32_t)v;
}

// The result, or the error code as an int.
PyObject* done(int rc, const Tensor& out)
{
    return rc ? PyLong_FromLong(rc) : THPVariable_Wrap(out);
}

void expect_args(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) refuse("expected ", want, " arguments, got ", n);
}

// x, W, bias, flags, residual, out, out_dtype, status, stream
PyObject* project(PyObject*, PyObject* const* o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 9);
    const Tensor &x = matrix(o[0], "x"), &W = matrix(o[1], "W");
    const Tensor *bias = optional_tensor(o[2], "bias"), *residual = optional_tensor(o[4], "residual");
    const Tensor *given = optional_tensor(o[5], "out"), *status = optional_tensor(o[7], "status");
    const at::Device dev = x.device();
    const int64_t T = x.size(0), K = x.size(1), N = W.size(0);
    const int64_t ldx = rows(x, "x", at::kBFloat16, T, K, dev), ldw = rows(W, "W", at::kBFloat16, N, K, dev);
    if (K > INT32_MAX || N > INT32_MAX) refuse("more than 2^31 - 1 columns or outputs");
    const at::ScalarType type = result_type(given, o[6]);
    const void* b = vector(bias, "bias", at::kBFloat16, N, dev);
    const int64_t ldr = residual ? rows(*residual, "residual", at::kBFloat16, T, N, dev) : 0;
    const int64_t ldy = given ? rows(*given, "out", type, T, N, dev) : N;
    int32_t* s = static_cast<int32_t*>(vector(status, "status", at::kInt, 1, dev));
    const uint32_t flags = flags_of(o[3]) | (type == at::kFloat ? ADAFUSE_OUT_F32 : 0u);
    On on(dev, o[8]);
    const Tensor out = given ? *given : at::empty({T, N}, x.options().dtype(type));
    return done(project_fn(x.data_ptr(), T, (int32_t)K, ldx, W.data_ptr(), (int32_t)N, ldw, b,
                           residual ? residual->data_ptr() : nullptr, ldr, out.data_ptr(), ldy, flags, s,
                           reinterpret_cast<adafuse_stream_t>(on.raw)), out);
    END_HANDLE_TH_ERRORS
}

// x, W_gate, W_up, bias_gate, bias_up, flags, out, status, stream
PyObject* gated_project(PyObject*, PyObject* const* o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 9);
    const Tensor &x = matrix(o[0], "x"), &Wg = matrix(o[1], "W_gate"), &Wu = matrix(o[2], "W_up");
    const Tensor *bias_gate = optional_tensor(o[3], "bias_gate"), *bias_up = optional_tensor(o[4], "bias_up");
    const Tensor *given = optional_tensor(o[6], "out"), *status = optional_tensor(o[7], "status");
    const at::Device dev = x.device();
    const int64_t T = x.size(0), K = x.size(1), N = Wg.size(0);
    const int64_t ldx = rows(x, "x", at::kBFloat16, T, K, dev), ldw = rows(Wg, "W_gate", at::kBFloat16, N, K, dev);
    if (rows(Wu, "W_up", at::kBFloat16, N, K, dev) != ldw && N > 1) refuse("W_gate and W_up need the same row stride");
    if (K > INT32_MAX || N > INT32_MAX) refuse("more than 2^31 - 1 columns or outputs");
    const void *bg = vector(bias_gate, "bias_gate", at::kBFloat16, N, dev);
    const void *bu = vector(bias_up, "bias_up", at::kBFloat16, N, dev);
    const int64_t ldy = given ? rows(*given, "out", at::kBFloat16, T, N, dev) : N;
    int32_t* s = static_cast<int32_t*>(vector(status, "status", at::kInt, 1, dev));
    const uint32_t flags = flags_of(o[5]);
    On on(dev, o[8]);
    const Tensor out = given ? *given : at::empty({T, N}, x.options());
    return done(gated_fn(x.data_ptr(), T, (int32_t)K, ldx, Wg.data_ptr(), Wu.data_ptr(), (int32_t)N, ldw, bg, bu,
                         out.data_ptr(), ldy, flags, s, reinterpret_cast<adafuse_stream_t>(on.raw)), out);
    END_HANDLE_TH_ERRORS
}

// y, bias, flags, up, residual, out, out_dtype, stream
PyObject* epilogue(PyObject*, PyObject* const* o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 8);
    const Tensor& y = matrix(o[0], "y");
    const Tensor *bias = optional_tensor(o[1], "bias"), *up = optional_tensor(o[3], "up");
    const Tensor *residual = optional_tensor(o[4], "residual"), *given = optional_tensor(o[5], "out");
    const at::Device dev = y.device();
    const int64_t T = y.size(0), N = y.size(1);
    const at::ScalarType in = y.scalar_type() == at::kFloat ? at::kFloat : at::kBFloat16;
    const int64_t ldy = rows(y, "y", in, T, N, dev);
    const at::ScalarType type = result_type(given, o[6]);
    const void* b = vector(bias, "bias", at::kBFloat16, N, dev);
    const int64_t ldu = up ? rows(*up, "up", in, T, N, dev) : 0;
    const int64_t ldr = residual ? rows(*residual, "residual", at::kBFloat16, T, N, dev) : 0;
    const int64_t ldo = given ? rows(*given, "out", type, T, N, dev) : N;
    const uint32_t flags = flags_of(o[2]) | (in == at::kFloat ? ADAFUSE_IN_F32 : 0u) |
                           (type == at::kFloat ? ADAFUSE_OUT_F32 : 0u);
    On on(dev, o[7]);
    const Tensor out = given ? *given : at::empty({T, N}, y.options().dtype(type));
    return done(epilogue_fn(y.data_ptr(), T, N, ldy, b, up ? up->data_ptr() : nullptr, ldu,
                            residual ? residual->data_ptr() : nullptr, ldr, out.data_ptr(), ldo, flags,
                            reinterpret_cast<adafuse_stream_t>(on.raw)), out);
    END_HANDLE_TH_ERRORS
}

adafuse_heads heads_of(const Tensor& t, const Tensor& out, const Tensor* weight, const char* name, const char* out_name,
                       const char* weight_name, int64_t T, int64_t D, at::Device dev)
{
    for (const Tensor* m : {&t, &out}) {
        const char* what = m == &t ? name : out_name;
        if (m->dim() != 3 || m->size(0) != T || m->size(1) != t.size(1) || m->size(2) != D ||
            m->scalar_type() != at::kBFloat16 || m->device() != dev)
            refuse(what, ": expected bfloat16 [", T, ", heads, ", D, "] on ", dev, ", got ", m->scalar_type(), " ",
                   m->sizes(), " on ", m->device());
        if (m->stride(2) != 1 && D > 1)
            refuse(what, ": the elements of a head must be adjacent (strides ", m->strides(), ")");
    }
    if (t.size(1) > INT32_MAX || D > INT32_MAX) refuse("more than 2^31 - 1 heads or elements");
    return adafuse_heads{t.data_ptr(), out.data_ptr(), t.stride(0), t.stride(1), out.stride(0), out.stride(1),
                         vector(weight, weight_name, at::kBFloat16, D, dev), (int32_t)t.size(1)};
}

// q, k, positions, freq, flags, factor, q_weight, k_weight, eps, q_out, k_out, stream
PyObject* rotary(PyObject*, PyObject* const* o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 12);
    const Tensor &q = tensor(o[0], "q"), &positions = tensor(o[2], "positions"), &freq = tensor(o[3], "freq");
    const Tensor *k = optional_tensor(o[1], "k"), *q_weight = optional_tensor(o[6], "q_weight");
    const Tensor *k_weight = optional_tensor(o[7], "k_weight"), *q_given = optional_tensor(o[9], "q_out");
    const Tensor* k_given = optional_tensor(o[10], "k_out");
    if (q.dim() != 3 || (k && k->dim() != 3)) refuse("q and k have three dimensions: tokens, heads, elements");
    if (!k && (k_weight || k_given)) refuse("k_weight and k_out go with k");
    const at::Device dev = q.device();
    const int64_t T = q.size(0), D = q.size(2);
    const bool narrow = positions.scalar_type() == at::kInt;
    const void* p = vector(&positions, "positions", narrow ? at::kInt : at::kLong, T, dev);
    if (freq.dim() != 1) refuse("freq has one dimension");
    const int64_t pairs = freq.size(0);
    const void* f = vector(&freq, "freq", at::kDouble, pairs, dev);
    if (pairs > INT32_MAX / 2) refuse("more frequencies than a head can have");
    const uint32_t flags = flags_of(o[4]) | (narrow ? ADAFUSE_POS_I32 : 0u);
    const double factor = PyFloat_AsDouble(o[5]), eps = PyFloat_AsDouble(o[8]);
    if (PyErr_Occurred()) throw python_error();
    On on(dev, o[11]);
    const Tensor q_out = q_given ? *q_given : at::empty(q.sizes(), q.options());
    const Tensor k_out = k_given ? *k_given : k ? at::empty(k->sizes(), k->options()) : Tensor();
    const adafuse_heads hq = heads_of(q, q_out, q_weight, "q", "q_out", "q_weight", T, D, dev);
    adafuse_heads hk;
    if (k) hk = heads_of(*k, k_out, k_weight, "k", "k_out", "k_weight", T, D, dev);
    const int rc = rotary_fn(&hq, k ? &hk : nullptr, T, (int32_t)D, (int32_t)(2 * pairs), p,
                             static_cast<const double*>(f), (float)factor, (float)eps, flags,
                             reinterpret_cast<adafuse_stream_t>(on.raw));
    if (rc) return PyLong_FromLong(rc);
    THPObjectPtr a(THPVariable_Wrap(q_out)), b(k ? THPVariable_Wrap(k_out) : Py_NewRef(Py_None));
    return PyTuple_Pack(2, a.get(), b.get());
    END_HANDLE_TH_ERRORS
}

// The addresses of the C ABI's entry points, in the order of the declarations above.
PyObject* install(PyObject*, PyObject* const* o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 4);
    void* at[4];
    for (int i = 0; i < 4; ++i) at[i] = PyLong_AsVoidPtr(o[i]);
    if (PyErr_Occurred()) throw python_error();
    project_fn = reinterpret_cast<decltype(project_fn)>(at[0]);
    gated_fn = reinterpret_cast<decltype(gated_fn)>(at[1]);
    epilogue_fn = reinterpret_cast<decltype(epilogue_fn)>(at[2]);
    rotary_fn = reinterpret_cast<decltype(rotary_fn)>(at[3]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

template <typename F>
PyCFunction as_method(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"install", as_method(install), METH_FASTCALL, nullptr},
    {"project", as_method(project), METH_FASTCALL, nullptr},
    {"gated_project", as_method(gated_project), METH_FASTCALL, nullptr},
    {"epilogue", as_method(epilogue), METH_FASTCALL, nullptr},
    {"rotary", as_method(rotary), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding() { return PyModule_Create(&module); }
