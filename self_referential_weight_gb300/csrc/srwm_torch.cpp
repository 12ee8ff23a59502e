// srwm_torch.cpp -- the PyTorch side of the linear attention and group norm
// entry points: a CPython module that checks tensors, allocates the outputs
// that the caller does not pass, and calls the C ABI of include/srwm.h on the
// tensors' device's current stream.  It holds no arithmetic.  A call of a few
// microseconds on the GPU would wait for its marshalling in Python; here that
// takes about as long as the launch itself.
//
// Every function takes its arguments by position, None for what is not given
// (binding.py documents them).  A non-zero status raises the class given to
// set_error, called with (status, name).
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "srwm.h"

namespace {

PyObject* g_error = nullptr;

const at::Tensor& tensor(PyObject* o, const char* name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor& t, const char* name)
{
    switch (t.scalar_type()) {
    case at::kFloat: return SRWM_F32;
    case at::kBFloat16: return SRWM_BF16;
    case at::kHalf: return SRWM_F16;
    default: TORCH_CHECK_VALUE(false, name, " must be float32, bfloat16 or float16");
    }
    return -1;
}

// The address of a contiguous CUDA tensor of this shape and type (null when empty).
void* address(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.is_cuda() && t.is_contiguous(), name, " must be a contiguous ",
                      c10::toString(type), " CUDA tensor");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    return t.numel() ? t.data_ptr() : nullptr;
}

void* address(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type)
{
    return address(tensor(o, name), name, shape, type);
}

void* optional(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type)
{
    return o == Py_None ? nullptr : address(o, name, shape, type);
}

// The caller's output tensor, checked, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    if (o == Py_None) return at::empty(shape, like.options().dtype(type));
    const at::Tensor& t = tensor(o, name);
    address(t, name, shape, type);
    return t;
}

void* data(const at::Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }

at::Tensor scratch(PyObject* o, size_t need, const at::Tensor& like)
{
    if (o == Py_None)
        return at::empty({static_cast<int64_t>(need > 16 ? need : 16)}, like.options().dtype(at::kByte));
    const at::Tensor& t = tensor(o, "workspace");
    TORCH_CHECK_VALUE(t.is_cuda() && t.is_contiguous(), "workspace must be a contiguous CUDA tensor");
    return t;
}

// Tokens of [B, T, H, d] (or [B, H, d]) tensors that lie one common distance apart: that distance in elements.
int64_t token_distance(std::initializer_list<std::pair<const at::Tensor*, const char*>> ts, at::IntArrayRef shape,
                       at::ScalarType type)
{
    const int64_t H = shape[shape.size() - 2], d = shape[shape.size() - 1];
    const int64_t B = shape[0], T = shape.size() == 4 ? shape[1] : 1;
    int64_t ld = -1;
    for (const auto& p : ts) {
        const at::Tensor& t = *p.first;
        TORCH_CHECK_VALUE(t.scalar_type() == type && t.is_cuda(), p.second, " must be a ", c10::toString(type),
                          " CUDA tensor");
        TORCH_CHECK_VALUE(t.sizes() == shape, p.second, " has shape ", t.sizes(), ", expected ", shape);
        if (t.numel() == 0) continue;
        const at::IntArrayRef st = t.strides();
        const int64_t mine = B * T == 1 ? H * d : T > 1 ? st[1] : st[0];
        TORCH_CHECK_VALUE((d == 1 || st[st.size() - 1] == 1) && (H == 1 || st[st.size() - 2] == d) &&
                              (T == 1 || B == 1 || st[0] == T * mine),
                          p.second, ": a token's heads must be contiguous and its tokens evenly spaced");
        TORCH_CHECK_VALUE(ld < 0 || ld == mine, p.second, " must have the strides of the tensors that go with it");
        ld = mine;
    }
    return ld < 0 ? H * d : ld;
}

const int* lengths_address(PyObject* o, int64_t B)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, "lengths");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.is_cuda() && t.is_contiguous() && t.dim() == 1 && t.size(0) == B,
                      "lengths must be a contiguous int32 CUDA tensor of ", B, " values");
    return static_cast<const int*>(data(t));
}

float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(v);
}

float scale_of(PyObject* o, int64_t d)
{
    return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : number(o);
}

long long integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int as_int(int64_t v) { return v > 0x7fffffff ? -1 : static_cast<int>(v); }   // the library refuses what does not fit

void* stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

void four(const at::Tensor& t, const char* name, int64_t dims)
{
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must have ", dims, " dimensions");
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
}

// The outputs as a tuple, or the status as an exception.
PyObject* finish(int status, const char* where, std::initializer_list<at::Tensor> outs)
{
    if (status != SRWM_OK) {
        PyObject* e = g_error ? PyObject_CallFunction(g_error, "is", status, where) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, where);
        }
        return nullptr;
    }
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
    Py_ssize_t i = 0;
    for (const at::Tensor& t : outs) PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(t));
    return tuple;
}

void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// q, k, v, log_decay, scale, S_init, lengths, o, S_final, workspace
PyObject* linattn_forward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 10);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int code = dtype_code(q, "q");
    four(q, "q", 4);
    const int64_t B = q.size(0), T = q.size(1), H = q.size(2), d = q.size(3);
    const int64_t ld = token_distance({{&q, "q"}, {&k, "k"}, {&v, "v"}}, q.sizes(), q.scalar_type());
    const int64_t decay[] = {H}, state[] = {B, H, d, d};
    const at::Tensor o = output(a[7], "o", q.sizes(), q.scalar_type(), q);
    const at::Tensor S = output(a[8], "S_final", state, at::kFloat, q);
    const int b = as_int(B), t = as_int(T), h = as_int(H), w = as_int(d);
    const at::Tensor ws = scratch(a[9], srwm_linattn_workspace_bytes(b, t, h, w), q);
    const int rc = srwm_linattn_forward(
        data(q), data(k), data(v), ld, static_cast<const float*>(address(a[3], "log_decay", decay, at::kFloat)),
        static_cast<const float*>(optional(a[5], "S_init", state, at::kFloat)), lengths_address(a[6], B), code, b, t, h, w,
        scale_of(a[4], d), data(o), static_cast<float*>(data(S)), ws.data_ptr(), ws.nbytes(), stream_of(q));
    return finish(rc, "srwm_linattn_forward", {o, S});
    END_HANDLE_TH_ERRORS
}

// q_t, k_t, v_t, log_decay, S_in, scale, o_t, S_out
PyObject* linattn_step(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 8);
    const at::Tensor &q = tensor(a[0], "q_t"), &k = tensor(a[1], "k_t"), &v = tensor(a[2], "v_t");
    const int code = dtype_code(q, "q_t");
    four(q, "q_t", 3);
    const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
    const int64_t ld = token_distance({{&q, "q_t"}, {&k, "k_t"}, {&v, "v_t"}}, q.sizes(), q.scalar_type());
    const int64_t decay[] = {H}, state[] = {B, H, d, d};
    const at::Tensor o = output(a[6], "o_t", q.sizes(), q.scalar_type(), q);
    const at::Tensor S = output(a[7], "S_out", state, at::kFloat, q);
    const int rc = srwm_linattn_step(data(q), data(k), data(v), ld,
                                     static_cast<const float*>(address(a[3], "log_decay", decay, at::kFloat)),
                                     static_cast<const float*>(address(a[4], "S_in", state, at::kFloat)), code, as_int(B),
                                     as_int(H), as_int(d), scale_of(a[5], d), data(o), static_cast<float*>(data(S)),
                                     stream_of(q));
    return finish(rc, "srwm_linattn_step", {o, S});
    END_HANDLE_TH_ERRORS
}

// q, k, v, log_decay, do, scale, S_init, lengths, dS_final, dq, dk, dv, dS_init, workspace
PyObject* linattn_backward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 14);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const int code = dtype_code(q, "q");
    four(q, "q", 4);
    const int64_t B = q.size(0), T = q.size(1), H = q.size(2), d = q.size(3);
    const int64_t ld = token_distance({{&q, "q"}, {&k, "k"}, {&v, "v"}}, q.sizes(), q.scalar_type());
    const int64_t decay[] = {H}, state[] = {B, H, d, d};
    const int given = (a[9] != Py_None) + (a[10] != Py_None) + (a[11] != Py_None);
    TORCH_CHECK_VALUE(given == 0 || given == 3, "dq, dk and dv: give all three or none");
    auto grad = [&](PyObject* o, const char* name) {
        return given ? tensor(o, name) : at::empty(q.sizes(), q.options());
    };
    const at::Tensor dq = grad(a[9], "dq"), dk = grad(a[10], "dk"), dv = grad(a[11], "dv");
    const int64_t ldg = token_distance({{&dq, "dq"}, {&dk, "dk"}, {&dv, "dv"}}, q.sizes(), q.scalar_type());
    const at::Tensor d0 = output(a[12], "dS_init", state, at::kFloat, q);
    const int b = as_int(B), t = as_int(T), h = as_int(H), w = as_int(d);
    const at::Tensor ws = scratch(a[13], srwm_linattn_backward_workspace_bytes(b, t, h, w), q);
    const int rc = srwm_linattn_backward(
        data(q), data(k), data(v), ld, static_cast<const float*>(address(a[3], "log_decay", decay, at::kFloat)),
        static_cast<const float*>(optional(a[6], "S_init", state, at::kFloat)), lengths_address(a[7], B), code, b, t, h, w,
        scale_of(a[5], d), address(a[4], "do", q.sizes(), q.scalar_type()),
        static_cast<const float*>(optional(a[8], "dS_final", state, at::kFloat)), data(dq), data(dk), data(dv), ldg,
        static_cast<float*>(data(d0)), ws.data_ptr(), ws.nbytes(), stream_of(q));
    return finish(rc, "srwm_linattn_backward", {dq, dk, dv, d0});
    END_HANDLE_TH_ERRORS
}

// x, gamma, beta, groups, eps, activation, y, mean, rstd, workspace
PyObject* groupnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 10);
    const float eps = number(a[4]);
    const at::Tensor& x = tensor(a[0], "x");
    const int code = dtype_code(x, "x");
    four(x, "x", 3);
    const int64_t N = x.size(0), L = x.size(1), C = x.size(2), G = integer(a[3]);
    TORCH_CHECK_VALUE(G > 0, "groups must be positive");
    const int64_t channels[] = {C}, stats[] = {N, G};
    const void* px = address(x, "x", x.sizes(), x.scalar_type());
    const at::Tensor y = output(a[6], "y", x.sizes(), x.scalar_type(), x);
    const at::Tensor mean = output(a[7], "mean", stats, at::kFloat, x), rstd = output(a[8], "rstd", stats, at::kFloat, x);
    const at::Tensor ws = scratch(a[9], srwm_groupnorm_workspace_bytes(N, L, as_int(C), as_int(G)), x);
    const int rc = srwm_groupnorm_forward(
        px, static_cast<const float*>(optional(a[1], "gamma", channels, at::kFloat)),
        static_cast<const float*>(optional(a[2], "beta", channels, at::kFloat)), code, N, L, as_int(C), as_int(G),
        eps, static_cast<int>(integer(a[5])), data(y), static_cast<float*>(data(mean)),
        static_cast<float*>(data(rstd)), ws.data_ptr(), ws.nbytes(), stream_of(x));
    return finish(rc, "srwm_groupnorm_forward", {y, mean, rstd});
    END_HANDLE_TH_ERRORS
}

// x, gamma, beta, groups, mean, rstd, dy, activation, dx, dgamma, dbeta, workspace
PyObject* groupnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 12);
    const at::Tensor& x = tensor(a[0], "x");
    const int code = dtype_code(x, "x");
    four(x, "x", 3);
    const int64_t N = x.size(0), L = x.size(1), C = x.size(2), G = integer(a[3]);
    TORCH_CHECK_VALUE(G > 0, "groups must be positive");
    const int64_t channels[] = {C}, stats[] = {N, G};
    const void* px = address(x, "x", x.sizes(), x.scalar_type());
    const at::Tensor dx = output(a[8], "dx", x.sizes(), x.scalar_type(), x);
    const at::Tensor dg = output(a[9], "dgamma", channels, at::kFloat, x), db = output(a[10], "dbeta", channels, at::kFloat, x);
    const at::Tensor ws = scratch(a[11], srwm_groupnorm_backward_workspace_bytes(N, L, as_int(C), as_int(G)), x);
    const int rc = srwm_groupnorm_backward(
        px, static_cast<const float*>(optional(a[1], "gamma", channels, at::kFloat)),
        static_cast<const float*>(optional(a[2], "beta", channels, at::kFloat)),
        static_cast<const float*>(address(a[4], "mean", stats, at::kFloat)),
        static_cast<const float*>(address(a[5], "rstd", stats, at::kFloat)), address(a[6], "dy", x.sizes(), x.scalar_type()),
        code, N, L, as_int(C), as_int(G), static_cast<int>(integer(a[7])), data(dx), static_cast<float*>(data(dg)),
        static_cast<float*>(data(db)), ws.data_ptr(), ws.nbytes(), stream_of(x));
    return finish(rc, "srwm_groupnorm_backward", {dx, dg, db});
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls)
{
    Py_XINCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"linattn_forward", fast(linattn_forward), METH_FASTCALL, nullptr},
    {"linattn_step", fast(linattn_step), METH_FASTCALL, nullptr},
    {"linattn_backward", fast(linattn_backward), METH_FASTCALL, nullptr},
    {"groupnorm_forward", fast(groupnorm_forward), METH_FASTCALL, nullptr},
    {"groupnorm_backward", fast(groupnorm_backward), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_srwm_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__srwm_torch() { return PyModule_Create(&module); }
