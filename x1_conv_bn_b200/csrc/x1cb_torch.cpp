// Marshalling of the floating-point calls' ordinary form in C++: tensors in, new
// tensors out, on the current stream of the current device.  In Python the
// checks and conversions of such a call take twice as long as the library's own
// part of it (allocation, argument checks, launch).  Every function returns None
// when anything is out of the ordinary -- an operand that is missing, on another
// device, strided, without storage, of another type or size, one that requires
// grad, or a call that the library refuses -- and the binding then takes its own way, which names what is
// wrong.  C++ exceptions (no memory for a result) leave as their Python ones.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/x1cb.h"

namespace {

// An operand, or NULL for None; `ok` turns false when it is out of the ordinary.
const at::Tensor *operand(PyObject *o, bool &ok, bool optional = false)
{
    if (optional && o == Py_None)
        return nullptr;
    if (!THPVariable_CheckExact(o)) {
        ok = false;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}

// A CUDA tensor with sizes, strides and memory of its own (not sparse, nested or
// the handle of a function transform).
bool on_gpu(const at::Tensor *t)
{
    return t->is_cuda() && t->layout() == at::kStrided && !t->is_nested() && t->has_storage();
}

// (the calls have no backward pass: one that autograd would record is refused)
bool plain(const at::Tensor *t, at::ScalarType type, int device)
{
    return on_gpu(t) && !(t->requires_grad() && at::GradMode::is_enabled()) && t->get_device() == device && t->scalar_type() == type && t->is_contiguous();
}

int dtype_code(at::ScalarType t)
{
    return t == at::kFloat ? X1CB_F32 : t == at::kBFloat16 ? X1CB_BF16 : t == at::kHalf ? X1CB_F16 : -1;
}

void *data(const at::Tensor *t) { return t ? t->data_ptr() : nullptr; }
template <typename T> T *data_as(const at::Tensor *t) { return static_cast<T *>(data(t)); }

bool sizes_are(const at::Tensor *t, at::IntArrayRef s) { return !t || t->sizes() == s; }

bool small(at::IntArrayRef s)
{
    for (int64_t n : s)
        if (n > INT_MAX)
            return false;
    return true;
}

PyObject *none() { return Py_NewRef(Py_None); }

// Runs a library call without the interpreter lock; true where it succeeded.
template <typename F> bool call(const F &f)
{
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = f();
    Py_END_ALLOW_THREADS;
    return status == X1CB_OK;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *t = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

at::Tensor scales_for(int64_t M, int64_t K, const at::TensorOptions &u8)
{
    return at::empty({(M + 127) / 128, (K + 127) / 128, 32, 16}, u8);
}

// norm(kind, x, gamma, beta, G, eps, r, act, q_mul), kind 0 same type, 1 int8, 2 MX4
PyObject *norm(PyObject *const *args, Py_ssize_t n)
{
    if (n != 9)
        return none();
    const long kind = PyLong_AsLong(args[0]), G = PyLong_AsLong(args[4]), act = PyLong_AsLong(args[7]);
    const double eps = PyFloat_AsDouble(args[5]), q_mul = PyFloat_AsDouble(args[8]);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    bool ok = G > 0 && G <= INT_MAX;
    const at::Tensor *x = operand(args[1], ok), *gamma = operand(args[2], ok, true);
    const at::Tensor *beta = operand(args[3], ok, true), *r = operand(args[6], ok, true);
    if (!ok || !on_gpu(x) || x->dim() != 4)
        return none();
    const int dev = x->get_device(), dt = dtype_code(x->scalar_type());
    const auto s = x->sizes();
    if (dt < 0 || dev != c10::cuda::current_device() || !plain(x, x->scalar_type(), dev) ||
        (gamma && !plain(gamma, at::kFloat, dev)) || (beta && !plain(beta, at::kFloat, dev)) ||
        (r && !plain(r, x->scalar_type(), dev)) || !small(s) || !sizes_are(gamma, {s[3]}) ||
        !sizes_are(beta, {s[3]}) || !sizes_are(r, s))
        return none();
    const int B = s[0], H = s[1], W = s[2], C = s[3];
    if (kind != 0 && C % 32)
        return none();
    at::AutoDispatchBelowADInplaceOrView guard;
    const auto u8 = x->options().dtype(at::kByte);
    at::Tensor y, sf, ws;
    if (kind == 0)
        y = at::empty(s, x->options());
    else if (kind == 1)
        y = at::empty({B, C / 32, H, W, 32}, x->options().dtype(at::kChar));
    else {
        y = at::empty({B, H, W, C / 2}, u8);
        sf = scales_for(static_cast<int64_t>(B) * H * W, C, u8);
    }
    const size_t need = group_norm_workspace_size(dt, B, H, W, C, static_cast<int>(G));
    if (need)
        ws = at::empty({static_cast<int64_t>(need)}, u8);
    void *stream = c10::cuda::getCurrentCUDAStream(dev).stream(), *w = need ? ws.data_ptr() : nullptr;
    const auto *g = data_as<float>(gamma), *b = data_as<float>(beta);
    const float e = static_cast<float>(eps);
    const bool done = call([&] {
        if (kind == 0)
            return group_norm_act(x->data_ptr(), dt, g, b, data(r), act, e, y.data_ptr(), w, need, B,
                                  H, W, C, G, stream);
        if (kind == 1)
            return group_norm_act_i8(x->data_ptr(), dt, g, b, data(r), act, e,
                                     static_cast<float>(q_mul), data_as<int8_t>(&y), w, need, B, H, W,
                                     C, G, stream);
        return group_norm_act_mx4(x->data_ptr(), dt, g, b, data(r), act, e, data_as<uint8_t>(&y),
                                  data_as<uint8_t>(&sf), w, need, B, H, W, C, G, stream);
    });
    if (!done)
        return none();
    return kind == 2 ? pair(y, sf) : THPVariable_Wrap(y);
}

// quantize(x)
PyObject *quantize(PyObject *const *args, Py_ssize_t n)
{
    bool ok = n == 1;
    const at::Tensor *x = ok ? operand(args[0], ok) : nullptr;
    if (!ok || !on_gpu(x) || x->dim() < 1)
        return none();
    const int dev = x->get_device(), dt = dtype_code(x->scalar_type());
    const int64_t K = x->size(-1);
    if (dt < 0 || dev != c10::cuda::current_device() || !plain(x, x->scalar_type(), dev) || K < 32 ||
        K % 32 || K > INT_MAX)
        return none();
    const int64_t M = x->numel() / K;
    at::AutoDispatchBelowADInplaceOrView guard;
    const auto u8 = x->options().dtype(at::kByte);
    auto shape = x->sizes().vec();
    shape.back() = K / 2;
    at::Tensor q = at::empty(shape, u8), sf = scales_for(M, K, u8);
    void *stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    if (!call([&] {
            return x1cb_quantize_mx4(x->data_ptr(), dt, data_as<uint8_t>(&q), data_as<uint8_t>(&sf), M,
                                     static_cast<int>(K), stream);
        }))
        return none();
    return pair(q, sf);
}

bool dtype_of(long code, at::ScalarType &t)
{
    t = code == X1CB_F32 ? at::kFloat : code == X1CB_BF16 ? at::kBFloat16 : at::kHalf;
    return code >= X1CB_F32 && code <= X1CB_F16;
}

bool scales_are(const at::Tensor *t, int64_t M, int64_t K)
{
    return t->sizes() == at::IntArrayRef({(M + 127) / 128, (K + 127) / 128, 32, 16});
}

// dequantize(codes, scales, dtype code)
PyObject *dequantize(PyObject *const *args, Py_ssize_t n)
{
    bool ok = n == 3;
    const long dt = ok ? PyLong_AsLong(args[2]) : -1;
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    at::ScalarType type;
    const at::Tensor *q = ok ? operand(args[0], ok) : nullptr, *sf = ok ? operand(args[1], ok) : nullptr;
    if (!ok || !dtype_of(dt, type) || !on_gpu(q) || q->dim() < 1)
        return none();
    const int dev = q->get_device();
    const int64_t K = 2 * q->size(-1);
    if (dev != c10::cuda::current_device() || !plain(q, at::kByte, dev) || !plain(sf, at::kByte, dev) ||
        K < 32 || K % 32 || K > INT_MAX)
        return none();
    const int64_t M = q->numel() / (K / 2);
    if (!scales_are(sf, M, K))
        return none();
    at::AutoDispatchBelowADInplaceOrView guard;
    auto shape = q->sizes().vec();
    shape.back() = K;
    at::Tensor x = at::empty(shape, q->options().dtype(type));
    void *stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    if (!call([&] {
            return x1cb_dequantize_mx4(data_as<uint8_t>(q), data_as<uint8_t>(sf), x.data_ptr(), dt, M,
                                       static_cast<int>(K), stream);
        }))
        return none();
    return THPVariable_Wrap(x);
}

// conv1x1(x, xs, w, ws, bias, r, act, dtype code)
PyObject *conv1x1(PyObject *const *args, Py_ssize_t n)
{
    bool ok = n == 8;
    const long act = ok ? PyLong_AsLong(args[6]) : -1, dt = ok ? PyLong_AsLong(args[7]) : -1;
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return none();
    }
    at::ScalarType type;
    if (!ok || !dtype_of(dt, type))
        return none();
    const at::Tensor *x = operand(args[0], ok), *xs = operand(args[1], ok), *w = operand(args[2], ok);
    const at::Tensor *ws = operand(args[3], ok), *bias = operand(args[4], ok, true);
    const at::Tensor *r = operand(args[5], ok, true);
    if (!ok || !on_gpu(x) || !on_gpu(w) || x->dim() != 4 || w->dim() != 2)
        return none();
    const int dev = x->get_device();
    if (dev != c10::cuda::current_device() || !plain(x, at::kByte, dev) || !plain(xs, at::kByte, dev) ||
        !plain(w, at::kByte, dev) || !plain(ws, at::kByte, dev) ||
        (bias && !plain(bias, at::kFloat, dev)) || (r && !plain(r, type, dev)))
        return none();
    const auto s = x->sizes();
    const int64_t half = s[3], N = w->size(0), M = s[0] * s[1] * s[2];
    const int64_t os[4] = {s[0], s[1], s[2], N};
    if (!small(s) || N > INT_MAX || half > INT_MAX / 2 || w->size(1) != half ||
        !scales_are(xs, M, 2 * half) || !scales_are(ws, N, 2 * half) || !sizes_are(bias, {N}) ||
        !sizes_are(r, os))
        return none();
    at::AutoDispatchBelowADInplaceOrView guard;
    at::Tensor out = at::empty(os, x->options().dtype(type));
    void *stream = c10::cuda::getCurrentCUDAStream(dev).stream();
    if (!call([&] {
            return conv1x1_bias_add_act_mx4(
                data_as<uint8_t>(x), data_as<uint8_t>(xs), data_as<uint8_t>(w), data_as<uint8_t>(ws),
                data_as<float>(bias), data(r), act, out.data_ptr(), dt, s[0], s[1], s[2],
                static_cast<int>(2 * half), static_cast<int>(N), stream);
        }))
        return none();
    return THPVariable_Wrap(out);
}

// raises(what), for tests: an allocation of `what` bytes of host memory, or the
// address of tensor `what`.
PyObject *raises(PyObject *const *args, Py_ssize_t n)
{
    if (n == 1 && THPVariable_CheckExact(args[0])) {
        THPVariable_Unpack(args[0]).data_ptr();
    } else if (n == 1) {
        const long long bytes = PyLong_AsLongLong(args[0]);
        if (PyErr_Occurred())
            return nullptr;
        at::empty({bytes}, at::TensorOptions().dtype(at::kByte));
    }
    return none();
}

// What Python calls: F, with its exceptions turned into Python's.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    return F(args, n);
    END_HANDLE_TH_ERRORS
}
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)> PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<F>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method<norm>("norm"),
                         method<quantize>("quantize"),
                         method<dequantize>("dequantize"),
                         method<conv1x1>("conv1x1"),
                         method<raises>("raises"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_x1cb_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__x1cb_torch(void)
{
    PyObject *m = PyModule_Create(&module);
    // (the build looks this text up: another torch or Python needs another module)
    if (m && PyModule_AddStringConstant(m, "built_for", X1CB_BUILT_FOR) < 0)
        Py_CLEAR(m);
    return m;
}
