// srwm_torch.cpp -- the PyTorch side of the operators' entry points (linear
// attention, group norm, short convolution, selective scan, RMS norm): a CPython module that checks tensors, allocates the outputs
// that the caller does not pass, and calls the C ABI of include/srwm.h on the
// tensors' device's current stream.  It holds no arithmetic.  A call of a few
// microseconds on the GPU would wait for its marshalling in Python; here that
// takes about as long as the launch itself.
//
// Every function takes its arguments by position, None for what is not given
// (binding.py documents them).  A non-zero status raises the class given to
// set_error, called with (status, name).
#include <Python.h>

#include <ATen/core/DimVector.h>
#include <ATen/cuda/EmptyTensor.h>
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

// A new tensor beside `like`, straight from the allocator: through the dispatcher it takes as long as a launch.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// The caller's output tensor, checked, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    if (o == Py_None) return fresh(shape, type, like);
    const at::Tensor& t = tensor(o, name);
    address(t, name, shape, type);
    return t;
}

void* data(const at::Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }
float* floats(const at::Tensor& t) { return static_cast<float*>(data(t)); }

at::Tensor scratch(PyObject* o, size_t need, const at::Tensor& like)
{
    if (o == Py_None)
        return fresh({static_cast<int64_t>(need > 16 ? need : 16)}, at::kByte, like);
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

// Elements between the rows of a [B, T, D] (or [B, D]) tensor whose rows are contiguous and evenly spaced.
int64_t row_distance(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.is_cuda(), name, " must be a ", c10::toString(type), " CUDA tensor");
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    const int64_t B = shape[0], T = shape.size() == 3 ? shape[1] : 1, D = shape[shape.size() - 1];
    if (t.numel() == 0 || B * T == 1) {
        TORCH_CHECK_VALUE(t.numel() == 0 || D == 1 || t.stride(-1) == 1, name, ": a token's channels must be contiguous");
        return D;
    }
    const at::IntArrayRef st = t.strides();
    const int64_t ld = T > 1 ? st[1] : st[0];
    TORCH_CHECK_VALUE((D == 1 || st[st.size() - 1] == 1) && (T == 1 || B == 1 || st[0] == T * ld), name,
                      ": a token's channels must be contiguous and its tokens evenly spaced");
    return ld;
}

// The caller's output, whose rows may lie apart, or a new one.
at::Tensor row_output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    return o == Py_None ? fresh(shape, type, like) : tensor(o, name);
}

// The operator's own output where it is wanted, or an undefined tensor (None).
at::Tensor output_if(bool wanted, PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like)
{
    TORCH_CHECK_VALUE(wanted || o == Py_None, name, ": nothing of it goes out of this call");
    return wanted ? output(o, name, shape, type, like) : at::Tensor();
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

// The library refuses what does not fit: to either side, since what a cut leaves of a number below -2^31 can be one that it takes.
int as_int(int64_t v) { return v < 0 || v > 0x7fffffff ? -1 : static_cast<int>(v); }

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
    for (const at::Tensor& t : outs) {
        if (!t.defined()) Py_INCREF(Py_None);
        PyTuple_SET_ITEM(tuple, i++, t.defined() ? THPVariable_Wrap(t) : Py_None);
    }
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
        return given ? tensor(o, name) : fresh(q.sizes(), q.scalar_type(), q);
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

// x, weight, bias, activation, state_init, lengths, y, state_final
PyObject* conv_forward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 8);
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const int code = dtype_code(x, "x");
    four(x, "x", 3);
    four(weight, "weight", 2);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2), W = weight.size(1);
    const int64_t taps[] = {D, W}, channels[] = {D}, state[] = {B, W > 0 ? W - 1 : 0, D};
    const int64_t ld = row_distance(x, "x", x.sizes(), x.scalar_type());
    const at::Tensor y = output(a[6], "y", x.sizes(), x.scalar_type(), x);
    const at::Tensor s = output(a[7], "state_final", state, x.scalar_type(), x);
    const int rc = srwm_conv_forward(
        data(x), ld, static_cast<const float*>(address(weight, "weight", taps, at::kFloat)),
        static_cast<const float*>(optional(a[2], "bias", channels, at::kFloat)), optional(a[4], "state_init", state, x.scalar_type()),
        lengths_address(a[5], B), code, as_int(B), as_int(T), as_int(D), as_int(W), static_cast<int>(integer(a[3])), data(y), data(s),
        stream_of(x));
    return finish(rc, "srwm_conv_forward", {y, s});
    END_HANDLE_TH_ERRORS
}

// x_t, weight, bias, state_in, activation, y_t, state_out
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 7);
    const at::Tensor &x = tensor(a[0], "x_t"), &weight = tensor(a[1], "weight");
    const int code = dtype_code(x, "x_t");
    four(x, "x_t", 2);
    four(weight, "weight", 2);
    const int64_t B = x.size(0), D = x.size(1), W = weight.size(1);
    const int64_t taps[] = {D, W}, channels[] = {D}, state[] = {B, W > 0 ? W - 1 : 0, D};
    const int64_t ld = row_distance(x, "x_t", x.sizes(), x.scalar_type());
    const void* in = address(a[3], "state_in", state, x.scalar_type());
    const at::Tensor y = output(a[5], "y_t", x.sizes(), x.scalar_type(), x);
    const at::Tensor s = output(a[6], "state_out", state, x.scalar_type(), x);
    const int rc = srwm_conv_step(data(x), ld, static_cast<const float*>(address(weight, "weight", taps, at::kFloat)),
                                  static_cast<const float*>(optional(a[2], "bias", channels, at::kFloat)), in, code, as_int(B),
                                  as_int(D), as_int(W), static_cast<int>(integer(a[4])), data(y), data(s), stream_of(x));
    return finish(rc, "srwm_conv_step", {y, s});
    END_HANDLE_TH_ERRORS
}

// x, weight, bias, dy, activation, state_init, lengths, dstate_final, dx, dweight, dbias, dstate_init, workspace
PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 13);
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const int code = dtype_code(x, "x");
    four(x, "x", 3);
    four(weight, "weight", 2);
    const int64_t B = x.size(0), T = x.size(1), D = x.size(2), W = weight.size(1);
    const int64_t taps[] = {D, W}, channels[] = {D}, state[] = {B, W > 0 ? W - 1 : 0, D};
    const int64_t ld = row_distance(x, "x", x.sizes(), x.scalar_type());
    const at::Tensor dx = row_output(a[8], "dx", x.sizes(), x.scalar_type(), x);
    const int64_t ldg = row_distance(dx, "dx", x.sizes(), x.scalar_type());
    const at::Tensor dw = output(a[9], "dweight", taps, at::kFloat, x);
    const at::Tensor db = output_if(a[2] != Py_None, a[10], "dbias", channels, at::kFloat, x);
    const at::Tensor d0 = output_if(a[5] != Py_None, a[11], "dstate_init", state, x.scalar_type(), x);
    const at::Tensor ws = scratch(a[12], srwm_conv_backward_workspace_bytes(as_int(B), as_int(T), as_int(D), as_int(W)), x);
    const int rc = srwm_conv_backward(
        data(x), ld, static_cast<const float*>(address(weight, "weight", taps, at::kFloat)),
        static_cast<const float*>(optional(a[2], "bias", channels, at::kFloat)), optional(a[5], "state_init", state, x.scalar_type()),
        lengths_address(a[6], B), code, as_int(B), as_int(T), as_int(D), as_int(W), static_cast<int>(integer(a[4])),
        address(a[3], "dy", x.sizes(), x.scalar_type()), optional(a[7], "dstate_final", state, x.scalar_type()), data(dx), ldg,
        floats(dw), floats(db), data(d0), ws.data_ptr(), ws.nbytes(), stream_of(x));
    return finish(rc, "srwm_conv_backward", {dx, dw, db, d0});
    END_HANDLE_TH_ERRORS
}

// What the selective scan's three calls have in common: u, dt, A, Bt, Ct, skip, z, dt_bias (of [B, T, ..], or of [B, ..]).
struct Scan {
    const at::Tensor& u;
    int code;
    int64_t B, T, D, N, G, ld_u, ld_dt, ld_z, ld_bc;
    const at::Tensor &dt, &Bt, &Ct;
    const float *A, *skip, *bias;
    const void* z;
    at::DimVector state, states, bc;   // [B, D, N], [D, N], the shape of B and C

    Scan(PyObject* pu, PyObject* pdt, PyObject* pA, PyObject* pB, PyObject* pC, PyObject* pskip, PyObject* pz, PyObject* pbias, bool one)
        : u(tensor(pu, one ? "u_t" : "u")), dt(tensor(pdt, one ? "dt_t" : "dt")), Bt(tensor(pB, one ? "B_t" : "Bt")), Ct(tensor(pC, one ? "C_t" : "Ct"))
    {
        code = dtype_code(u, "u");
        four(u, "u", one ? 2 : 3);
        four(Bt, "B", one ? 3 : 4);
        B = u.size(0), T = one ? 1 : u.size(1), D = u.size(-1), G = Bt.size(-2), N = Bt.size(-1);
        state = {B, D, N}, states = {D, N};
        bc = one ? at::DimVector{B, G, N} : at::DimVector{B, T, G, N};
        const int64_t channels[] = {D};
        ld_u = row_distance(u, "u", u.sizes(), u.scalar_type());
        ld_dt = row_distance(dt, "dt", u.sizes(), u.scalar_type());
        ld_bc = token_distance({{&Bt, "B"}, {&Ct, "C"}}, bc, u.scalar_type());
        A = static_cast<const float*>(address(pA, "A", states, at::kFloat));
        skip = static_cast<const float*>(optional(pskip, "skip", channels, at::kFloat));
        bias = static_cast<const float*>(optional(pbias, "dt_bias", channels, at::kFloat));
        z = nullptr, ld_z = D;
        if (pz != Py_None) {
            const at::Tensor& t = tensor(pz, "z");
            ld_z = row_distance(t, "z", u.sizes(), u.scalar_type());
            z = data(t);
        }
    }
};

// u, dt, A, Bt, Ct, skip, z, dt_bias, softplus, h_init, lengths, y, h_final, workspace
PyObject* ssm_forward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 14);
    const Scan s(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], false);
    const at::Tensor y = output(a[11], "y", s.u.sizes(), s.u.scalar_type(), s.u);
    const at::Tensor h = output(a[12], "h_final", s.state, at::kFloat, s.u);
    const int b = as_int(s.B), t = as_int(s.T), d = as_int(s.D), n = as_int(s.N), g = as_int(s.G);
    const at::Tensor ws = scratch(a[13], srwm_ssm_workspace_bytes(b, t, d, n, g), s.u);
    const int rc = srwm_ssm_forward(data(s.u), s.ld_u, data(s.dt), s.ld_dt, s.A, data(s.Bt), data(s.Ct), s.ld_bc, s.skip, s.z, s.ld_z,
                                    s.bias, static_cast<int>(integer(a[8])),
                                    static_cast<const float*>(optional(a[9], "h_init", s.state, at::kFloat)), lengths_address(a[10], s.B),
                                    s.code, b, t, d, n, g, data(y), floats(h), ws.data_ptr(), ws.nbytes(), stream_of(s.u));
    return finish(rc, "srwm_ssm_forward", {y, h});
    END_HANDLE_TH_ERRORS
}

// u_t, dt_t, A, B_t, C_t, h_in, skip, z_t, dt_bias, softplus, y_t, h_out
PyObject* ssm_step(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 12);
    const Scan s(a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], true);
    const float* in = static_cast<const float*>(address(a[5], "h_in", s.state, at::kFloat));
    const at::Tensor y = output(a[10], "y_t", s.u.sizes(), s.u.scalar_type(), s.u);
    const at::Tensor h = output(a[11], "h_out", s.state, at::kFloat, s.u);
    const int rc = srwm_ssm_step(data(s.u), s.ld_u, data(s.dt), s.ld_dt, s.A, data(s.Bt), data(s.Ct), s.ld_bc, s.skip, s.z, s.ld_z,
                                 s.bias, static_cast<int>(integer(a[9])), in, s.code, as_int(s.B), as_int(s.D), as_int(s.N),
                                 as_int(s.G), data(y), floats(h), stream_of(s.u));
    return finish(rc, "srwm_ssm_step", {y, h});
    END_HANDLE_TH_ERRORS
}

// u, dt, A, Bt, Ct, dy, skip, z, dt_bias, softplus, h_init, lengths, dh_final, du, ddt, dA, dB, dC, dskip, dz, ddt_bias,
// dh_init, workspace
PyObject* ssm_backward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 23);
    const Scan s(a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], false);
    const at::ScalarType type = s.u.scalar_type();
    const int64_t channels[] = {s.D};
    const bool gated = a[7] != Py_None;
    TORCH_CHECK_VALUE((a[16] == Py_None) == (a[17] == Py_None), "dB and dC: give both or none");
    const at::Tensor du = output(a[13], "du", s.u.sizes(), type, s.u), ddt = output(a[14], "ddt", s.u.sizes(), type, s.u);
    const at::Tensor dA = output(a[15], "dA", s.states, at::kFloat, s.u);
    const at::Tensor dB = row_output(a[16], "dB", s.bc, type, s.u), dC = row_output(a[17], "dC", s.bc, type, s.u);
    const int64_t ld_dbc = token_distance({{&dB, "dB"}, {&dC, "dC"}}, s.bc, type);
    const at::Tensor dskip = output_if(a[6] != Py_None, a[18], "dskip", channels, at::kFloat, s.u);
    TORCH_CHECK_VALUE(gated || a[19] == Py_None, "dz: there is no z");
    const at::Tensor dz = gated ? row_output(a[19], "dz", s.u.sizes(), type, s.u) : at::Tensor();
    const int64_t ld_dz = gated ? row_distance(dz, "dz", s.u.sizes(), type) : s.D;
    const at::Tensor dbias = output_if(a[8] != Py_None, a[20], "ddt_bias", channels, at::kFloat, s.u);
    const at::Tensor d0 = output_if(a[10] != Py_None, a[21], "dh_init", s.state, at::kFloat, s.u);
    const int b = as_int(s.B), t = as_int(s.T), d = as_int(s.D), n = as_int(s.N), g = as_int(s.G);
    const at::Tensor ws = scratch(a[22], srwm_ssm_backward_workspace_bytes(b, t, d, n, g), s.u);
    const int rc = srwm_ssm_backward(
        data(s.u), s.ld_u, data(s.dt), s.ld_dt, s.A, data(s.Bt), data(s.Ct), s.ld_bc, s.skip, s.z, s.ld_z, s.bias,
        static_cast<int>(integer(a[9])), static_cast<const float*>(optional(a[10], "h_init", s.state, at::kFloat)),
        lengths_address(a[11], s.B), s.code, b, t, d, n, g, address(a[5], "dy", s.u.sizes(), type),
        static_cast<const float*>(optional(a[12], "dh_final", s.state, at::kFloat)), data(du), data(ddt), floats(dA), data(dB),
        data(dC), ld_dbc, floats(dskip), data(dz), ld_dz, floats(dbias), floats(d0), ws.data_ptr(), ws.nbytes(), stream_of(s.u));
    return finish(rc, "srwm_ssm_backward", {du, ddt, dA, dB, dC, dskip, dz, dbias, d0});
    END_HANDLE_TH_ERRORS
}

// x, gamma, residual, eps, out, block, y, scale, total, rstd
PyObject* rmsnorm_forward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 10);
    const float eps = number(a[3]);
    const at::Tensor& x = tensor(a[0], "x");
    const int code = dtype_code(x, "x");
    four(x, "x", 2);
    const int out = static_cast<int>(integer(a[4]));
    const int64_t N = x.size(0), C = x.size(1), block = integer(a[5]);
    const bool e4m3 = out == SRWM_OUT_E4M3, added = a[2] != Py_None;
    const int64_t channels[] = {C}, rows[] = {N}, scales[] = {N, block > 0 ? C / block : 1};
    const void* px = address(x, "x", x.sizes(), x.scalar_type());
    const at::Tensor y = output(a[6], "y", x.sizes(), e4m3 ? at::kFloat8_e4m3fn : x.scalar_type(), x);
    const at::Tensor scale = output_if(e4m3, a[7], "scale", scales, at::kFloat, x);
    const at::Tensor total = output_if(added, a[8], "total", x.sizes(), x.scalar_type(), x);
    const at::Tensor rstd = output(a[9], "rstd", rows, at::kFloat, x);
    const int rc = srwm_rmsnorm_forward(px, optional(a[2], "residual", x.sizes(), x.scalar_type()),
                                        static_cast<const float*>(optional(a[1], "gamma", channels, at::kFloat)), code, N, as_int(C),
                                        eps, out, as_int(block), data(y), floats(scale), data(total), floats(rstd), stream_of(x));
    return finish(rc, "srwm_rmsnorm_forward", {y, scale, total, rstd});
    END_HANDLE_TH_ERRORS
}

// total, gamma, rstd, dy, dtotal, dx, dgamma, workspace
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t na)
{
    HANDLE_TH_ERRORS
    count(na, 8);
    const at::Tensor& x = tensor(a[0], "total");
    const int code = dtype_code(x, "total");
    four(x, "total", 2);
    const int64_t N = x.size(0), C = x.size(1);
    const int64_t channels[] = {C}, rows[] = {N};
    const void* px = address(x, "total", x.sizes(), x.scalar_type());
    const at::Tensor dx = output(a[5], "dx", x.sizes(), x.scalar_type(), x);
    const at::Tensor dg = output_if(a[1] != Py_None, a[6], "dgamma", channels, at::kFloat, x);
    const at::Tensor ws = scratch(a[7], srwm_rmsnorm_backward_workspace_bytes(N, as_int(C)), x);
    const int rc = srwm_rmsnorm_backward(px, static_cast<const float*>(optional(a[1], "gamma", channels, at::kFloat)),
                                         static_cast<const float*>(address(a[2], "rstd", rows, at::kFloat)),
                                         address(a[3], "dy", x.sizes(), x.scalar_type()), optional(a[4], "dtotal", x.sizes(), x.scalar_type()),
                                         code, N, as_int(C), data(dx), floats(dg), ws.data_ptr(), ws.nbytes(), stream_of(x));
    return finish(rc, "srwm_rmsnorm_backward", {dx, dg});
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
    {"conv_forward", fast(conv_forward), METH_FASTCALL, nullptr},
    {"conv_step", fast(conv_step), METH_FASTCALL, nullptr},
    {"conv_backward", fast(conv_backward), METH_FASTCALL, nullptr},
    {"ssm_forward", fast(ssm_forward), METH_FASTCALL, nullptr},
    {"ssm_step", fast(ssm_step), METH_FASTCALL, nullptr},
    {"ssm_backward", fast(ssm_backward), METH_FASTCALL, nullptr},
    {"rmsnorm_forward", fast(rmsnorm_forward), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", fast(rmsnorm_backward), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_srwm_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__srwm_torch() { return PyModule_Create(&module); }
