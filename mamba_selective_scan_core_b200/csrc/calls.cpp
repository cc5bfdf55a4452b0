// Python calls of the operators that a decoded token makes once per layer.
//
// A launch takes 2 to 3 us of host time; the same call through ctypes, with a
// dozen tensors looked at from Python, took 10 to 14.  Here the tensors are
// looked at where torch keeps them, the outputs come from torch's allocator,
// and the C entry point is called by its address (of whichever build of the
// library Python loaded).  A call that does not fit -- a tensor of another
// type, shape, device or layout, an argument that the library refuses --
// returns None without having launched anything, and the Python side takes its
// own path, which finds out what is wrong and says so.  A launch that fails,
// perhaps after others of the call, is raised here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mamba_mixer.h"

namespace {

struct Library {
    decltype(&mamba_gdr_fwd) gdr_fwd = nullptr;
    decltype(&mamba_gdr_workspace_size) gdr_workspace_size = nullptr;
    decltype(&mamba_gdr_state_update) gdr_state_update = nullptr;
    decltype(&mamba_proj_q4) proj_q4 = nullptr;
    PyObject* error = nullptr;        // MixerError(status, name)
} g_lib;

// A tensor argument: null when it is None, `bad` when it is anything else
// that is not plainly a tensor.
const at::Tensor* tensor(PyObject* o, bool& bad) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) {
        bad = true;
        return nullptr;
    }
    return &THPVariable_Unpack(o);
}
bool on(const at::Tensor& t, int dev, at::ScalarType type) {
    return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.layout() == at::kStrided;
}
bool dense(const at::Tensor* t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    return t && on(*t, dev, type) && t->sizes() == shape && t->is_contiguous();
}
bool dense_or_none(const at::Tensor* t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    return !t || dense(t, dev, type, shape);
}
// Elements between the rows of a [.., heads, width] tensor (tokens, or
// sequences and their tokens, before those) whose rows are dense and evenly
// spaced; -1 when they are not.  A dimension of one has no stride to go by.
int64_t row_stride(const at::Tensor* t, int dev, at::ScalarType type, at::IntArrayRef shape) {
    if (!t || !on(*t, dev, type) || t->sizes() != shape) return -1;
    const at::IntArrayRef st = t->strides();
    const size_t n = shape.size();
    if (st[n - 1] != 1 || (shape[n - 2] != 1 && st[n - 2] != shape[n - 1])) return -1;
    const int64_t tokens = shape[n - 3], seqs = n == 4 ? shape[0] : 1;
    if (tokens < 1) return -1;
    if (seqs == 1) return tokens > 1 ? st[n - 3] : shape[n - 2] * shape[n - 1];
    if (tokens == 1) return st[0];
    return st[0] == tokens * st[1] ? st[1] : -1;
}
const float* f32(const at::Tensor* t) { return t ? static_cast<const float*>(t->const_data_ptr()) : nullptr; }
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
bool number(PyObject* o, float dflt, float& out) {
    if (o == Py_None) {
        out = dflt;
        return true;
    }
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    out = static_cast<float>(v);
    return true;
}
PyObject* none() { Py_RETURN_NONE; }
// what a status other than MM_OK makes of a call
PyObject* failed(mm_status st, const char* name) {
    if (st != MM_ERR_CUDA) return none();     // refused before its first launch
    PyObject* e = PyObject_CallFunction(g_lib.error, "is", static_cast<int>(st), name);
    if (e) PyErr_SetObject(g_lib.error, e);
    Py_XDECREF(e);
    return nullptr;
}
bool activation(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }
mm_dtype code(at::ScalarType t) { return t == at::kBFloat16 ? MM_BF16 : MM_F32; }

// gdr_fwd(q, k, v, dt, beta, dt_bias, A, h0, scale, norm_eps, y, h_last, workspace) -> (y, h_last) or None
PyObject* gdr_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13 || !g_lib.gdr_fwd) return none();
    bool bad = false;
    const at::Tensor *q = tensor(a[0], bad), *k = tensor(a[1], bad), *v = tensor(a[2], bad), *dt = tensor(a[3], bad),
                     *beta = tensor(a[4], bad), *bias = tensor(a[5], bad), *A = tensor(a[6], bad), *h0 = tensor(a[7], bad),
                     *y = tensor(a[10], bad), *h_last = tensor(a[11], bad), *ws = tensor(a[12], bad);
    if (bad || !q || !v || v->dim() != 4 || q->dim() != 4 || !v->is_cuda()) return none();
    const int dev = v->get_device();
    const at::ScalarType type = v->scalar_type();
    const int64_t B = v->size(0), L = v->size(1), H = v->size(2), P = v->size(3), G = q->size(2), N = q->size(3);
    const int64_t qs = row_stride(q, dev, type, {B, L, G, N}), ks = row_stride(k, dev, type, {B, L, G, N}),
                  vs = row_stride(v, dev, type, {B, L, H, P});
    float scale, eps;
    if (!activation(type) || B < 1 || qs < 0 || ks < 0 || vs < 0 || !dense(dt, dev, type, {B, L, H}) ||
        !dense(beta, dev, type, {B, L, H}) || !dense(A, dev, at::kFloat, {H}) || !dense_or_none(bias, dev, at::kFloat, {H}) ||
        !dense_or_none(h0, dev, at::kFloat, {B, H, P, N}) || !dense_or_none(y, dev, type, {B, L, H, P}) ||
        !dense_or_none(h_last, dev, at::kFloat, {B, H, P, N}) || (ws && (!ws->is_cuda() || ws->get_device() != dev || !ws->is_contiguous())) ||
        !number(a[8], static_cast<float>(1.0 / std::sqrt(static_cast<double>(N))), scale) ||
        a[9] == Py_None || !number(a[9], 0.0f, eps))
        return none();
    const c10::cuda::OptionalCUDAGuard guard(v->device());
    at::Tensor y_new, h_new, ws_new;
    if (!y) y = &(y_new = empty({B, L, H, P}, type, *v));
    if (!h_last) h_last = &(h_new = empty({B, H, P, N}, at::kFloat, *v));
    if (!ws) {
        const int64_t bytes = static_cast<int64_t>(g_lib.gdr_workspace_size(B, L, H, P, N, G, code(type)));
        ws = &(ws_new = empty({std::max<int64_t>(bytes, 256)}, at::kByte, *v));
    }
    const mm_status st = g_lib.gdr_fwd(q->const_data_ptr(), k->const_data_ptr(), v->const_data_ptr(), dt->const_data_ptr(),
                                       beta->const_data_ptr(), f32(bias), f32(A), f32(h0), y->mutable_data_ptr(),
                                       static_cast<float*>(h_last->mutable_data_ptr()), B, L, G, H, P, N, qs, ks, vs, scale, eps,
                                       code(type), ws->mutable_data_ptr(), ws->nbytes(), c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != MM_OK) return failed(st, "mamba_gdr_fwd");
    PyObject* yo = y_new.defined() ? THPVariable_Wrap(y_new) : Py_NewRef(a[10]);
    PyObject* ho = h_new.defined() ? THPVariable_Wrap(h_new) : Py_NewRef(a[11]);
    PyObject* out = yo && ho ? PyTuple_Pack(2, yo, ho) : nullptr;
    Py_XDECREF(yo);
    Py_XDECREF(ho);
    return out;
}

// gdr_state_update(q, k, v, dt, beta, dt_bias, A, state, scale, norm_eps, y) -> y or None
PyObject* gdr_state_update(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 11 || !g_lib.gdr_state_update) return none();
    bool bad = false;
    const at::Tensor *q = tensor(a[0], bad), *k = tensor(a[1], bad), *v = tensor(a[2], bad), *dt = tensor(a[3], bad),
                     *beta = tensor(a[4], bad), *bias = tensor(a[5], bad), *A = tensor(a[6], bad), *state = tensor(a[7], bad),
                     *y = tensor(a[10], bad);
    if (bad || !q || !v || v->dim() != 3 || q->dim() != 3 || !v->is_cuda()) return none();
    const int dev = v->get_device();
    const at::ScalarType type = v->scalar_type();
    const int64_t B = v->size(0), H = v->size(1), P = v->size(2), G = q->size(1), N = q->size(2);
    const int64_t qs = row_stride(q, dev, type, {B, G, N}), ks = row_stride(k, dev, type, {B, G, N}),
                  vs = row_stride(v, dev, type, {B, H, P});
    float scale, eps;
    if (!activation(type) || B < 1 || qs < 0 || ks < 0 || vs < 0 || !dense(dt, dev, type, {B, H}) ||
        !dense(beta, dev, type, {B, H}) || !dense(A, dev, at::kFloat, {H}) || !dense_or_none(bias, dev, at::kFloat, {H}) ||
        !dense(state, dev, at::kFloat, {B, H, P, N}) || !dense_or_none(y, dev, type, {B, H, P}) ||
        !number(a[8], static_cast<float>(1.0 / std::sqrt(static_cast<double>(N))), scale) ||
        a[9] == Py_None || !number(a[9], 0.0f, eps))
        return none();
    const c10::cuda::OptionalCUDAGuard guard(v->device());
    at::Tensor y_new;
    if (!y) y = &(y_new = empty({B, H, P}, type, *v));
    const mm_status st = g_lib.gdr_state_update(
        q->const_data_ptr(), k->const_data_ptr(), v->const_data_ptr(), dt->const_data_ptr(), beta->const_data_ptr(), f32(bias), f32(A),
        static_cast<float*>(state->mutable_data_ptr()), y->mutable_data_ptr(), B, G, H, P, N, qs, ks, vs, scale, eps, code(type),
        c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != MM_OK) return failed(st, "mamba_gdr_state_update");
    return y_new.defined() ? THPVariable_Wrap(y_new) : Py_NewRef(a[10]);
}

// proj_q4(x, W, scales, zeros, group, out, bf16_out) -> out or None
PyObject* proj_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 7 || !g_lib.proj_q4) return none();
    bool bad = false;
    const at::Tensor *x = tensor(a[0], bad), *W = tensor(a[1], bad), *scales = tensor(a[2], bad), *zeros = tensor(a[3], bad),
                     *out = tensor(a[5], bad);
    const long group = PyLong_AsLong(a[4]);
    if (group <= 0) {
        PyErr_Clear();
        return none();
    }
    if (bad || !x || !W || x->dim() != 2 || W->dim() != 2 || !x->is_cuda()) return none();
    const int dev = x->get_device();
    const int64_t M = x->size(0), K = x->size(1), N = W->size(0);
    const at::ScalarType type = a[6] == Py_True ? at::kBFloat16 : at::kFloat;
    if (!dense(x, dev, at::kBFloat16, {M, K}) || !dense(W, dev, at::kByte, {N, K / 2}) ||
        !dense(scales, dev, at::kBFloat16, {N, K / group}) || !dense_or_none(zeros, dev, at::kBFloat16, {N, K / group}) ||
        !dense_or_none(out, dev, type, {M, N}))
        return none();
    const c10::cuda::OptionalCUDAGuard guard(x->device());
    at::Tensor made;
    if (!out) out = &(made = empty({M, N}, type, *x));
    const mm_status st = g_lib.proj_q4(x->const_data_ptr(), W->const_data_ptr(), scales->const_data_ptr(),
                                       zeros ? zeros->const_data_ptr() : nullptr, out->mutable_data_ptr(), M, N, K, group, code(type),
                                       c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != MM_OK) return failed(st, "mamba_proj_q4");
    return made.defined() ? THPVariable_Wrap(made) : Py_NewRef(a[5]);
}

// No C++ exception leaves an entry: torch's allocator may throw, and Python
// sees what it sees of torch's own calls (torch.OutOfMemoryError, ..).
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    return F(self, a, n);
    END_HANDLE_TH_ERRORS
}

// bind(gdr_fwd, gdr_workspace_size, gdr_state_update, proj_q4, error): the entry points' addresses, and the class of a failure
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes four addresses and an exception class");
        return nullptr;
    }
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_lib.gdr_fwd = reinterpret_cast<decltype(g_lib.gdr_fwd)>(p[0]);
    g_lib.gdr_workspace_size = reinterpret_cast<decltype(g_lib.gdr_workspace_size)>(p[1]);
    g_lib.gdr_state_update = reinterpret_cast<decltype(g_lib.gdr_state_update)>(p[2]);
    g_lib.proj_q4 = reinterpret_cast<decltype(g_lib.proj_q4)>(p[3]);
    Py_INCREF(a[4]);
    Py_XSETREF(g_lib.error, a[4]);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    {"gdr_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<gdr_fwd>)), METH_FASTCALL, nullptr},
    {"gdr_state_update", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<gdr_state_update>)), METH_FASTCALL, nullptr},
    {"proj_q4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<proj_q4>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", MM_CALLS_FOR, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
