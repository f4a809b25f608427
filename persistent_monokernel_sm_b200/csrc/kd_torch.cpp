// kd_torch.cpp -- the prompt operators on torch tensors, as the Python module _kd_torch: checks,
// allocation of the outputs and workspaces with torch's allocator, and the call into libkd on the
// current stream of the tensors' device. The same in Python takes 6 to 9 us a call, more than a
// token's products take on the GPU; here it takes 1 to 2. No autograd graph is recorded: where gradients are
// enabled, a tensor that requires them is refused.
//
// The functions take their arguments by position (operators.py, which documents them, gives names
// and defaults) and raise the package's KdError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "kd.h"

namespace {

PyObject* g_error = nullptr;  // KdError

struct Refused {};  // the Python error is set

[[noreturn]] void raise(int code, const char* text) {
    PyObject* e = PyObject_CallFunction(g_error, "is", code, text);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}
[[noreturn]] void refuse(const char* fmt, ...) {
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    raise(KD_EINVAL, text);
}
void check(int rc) {
    if (rc) raise(rc, kd_op_error());
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

const at::Tensor& tensor(const char* name, PyObject* o) {
    if (!THPVariable_Check(o)) refuse("%s must be a tensor: got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

struct Kind {  // of a call: its input type and device
    at::ScalarType type;
    int code, dev;
};

void no_graph_lost(const char* name, const at::Tensor& t) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse("%s requires grad, and no graph is recorded: call under torch.no_grad() or in an autograd.Function", name);
}

// torch's count of in-place changes, by which a backward pass notices that a value it needs is gone.
void changed(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The first input of `dim` dimensions, which sets type and device.
Kind kind_of(const char* name, const at::Tensor& t, int64_t dim) {
    no_graph_lost(name, t);
    if (t.dim() != dim || !t.is_cuda()) refuse("%s must be a %d-D CUDA tensor: got %s on %s", name, (int)dim, shape_of(t).c_str(), t.device().str().c_str());
    const auto type = t.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) refuse("%s must be bfloat16 or float16: got %s", name, c10::toString(type));
    return {type, type == at::kBFloat16 ? KD_BF16 : KD_F16, t.get_device()};
}

void same(const char* name, const at::Tensor& t, at::ScalarType type, int dev) {
    no_graph_lost(name, t);
    if (!t.is_cuda() || t.scalar_type() != type || t.get_device() != dev)
        refuse("%s must be a %s tensor on cuda:%d: got %s on %s", name, c10::toString(type), dev, c10::toString(t.scalar_type()), t.device().str().c_str());
}

// Checks a matrix; returns its row stride.
int64_t matrix(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, at::ScalarType type, int dev) {
    same(name, t, type, dev);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse("%s has shape %s, expected (%lld, %lld)", name, shape_of(t).c_str(), (long long)rows, (long long)cols);
    if (cols > 1 && t.stride(1) != 1) refuse("%s: the last dimension must be contiguous", name);
    return t.stride(0);
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

int act_id(PyObject* o) {
    if (o == Py_None) return KD_ACT_NONE;
    static const char* names[4] = {"none", "relu", "silu", "gelu"};
    if (PyUnicode_Check(o))
        for (int i = 0; i < 4; ++i)
            if (PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
    refuse("act must be one of none, relu, silu, gelu");
}

void args_of(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse("expected %d arguments, got %d", (int)want, (int)n);
}

// Runs f, and turns what it throws into the Python error: nothing leaves through Python's frames.
template <typename F>
PyObject* guarded(F f) {
    try {
        at::AutoDispatchBelowADInplaceOrView no_graph;
        return f();
    } catch (const Refused&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// linear(x, w, bias, act, residual, out, out_dtype, w_t)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        args_of(n_args, 8);
        const at::Tensor &x = tensor("x", a[0]), &w = tensor("w", a[1]);
        const Kind k = kind_of("x", x, 2);
        if (w.dim() != 2) refuse("w must be a 2-D tensor");
        kd_linear_args q{};
        q.w_transposed = PyObject_IsTrue(a[7]);
        if (q.w_transposed < 0) throw Refused();
        q.m = x.size(0), q.k = x.size(1), q.n = w.size(q.w_transposed ? 1 : 0);
        q.dtype = k.code;
        q.act = act_id(a[3]);
        q.x = x.data_ptr(), q.ld_x = matrix("x", x, q.m, q.k, k.type, k.dev);
        q.w = w.data_ptr();
        q.ld_w = q.w_transposed ? matrix("w", w, q.k, q.n, k.type, k.dev) : matrix("w", w, q.n, q.k, k.type, k.dev);
        at::ScalarType type = k.type;
        if (a[6] != Py_None) {
            if (!THPDtype_Check(a[6])) refuse("out_dtype must be a torch.dtype");
            type = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
        } else if (a[5] != Py_None) {
            type = tensor("out", a[5]).scalar_type();
        }
        if (type != k.type && type != at::kFloat) refuse("out_dtype must be %s or Float: got %s", c10::toString(k.type), c10::toString(type));
        q.out_dtype = type == at::kFloat ? KD_F32 : k.code;
        c10::cuda::OptionalCUDAGuard guard;
        if (k.dev != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)k.dev);
        if (a[2] != Py_None) {
            const at::Tensor& b = tensor("bias", a[2]);
            same("bias", b, k.type, k.dev);
            if (b.dim() != 1 || b.size(0) != q.n || (q.n > 1 && b.stride(0) != 1)) refuse("bias must be a contiguous (%lld,) tensor", (long long)q.n);
            q.bias = b.data_ptr();
        }
        if (a[4] != Py_None) {
            const at::Tensor& r = tensor("residual", a[4]);
            q.ld_residual = matrix("residual", r, q.m, q.n, type, k.dev);
            q.residual = r.data_ptr();
        }
        at::Tensor fresh;
        if (a[5] == Py_None) {
            fresh = empty({q.m, q.n}, type, k.dev);
            q.out = fresh.data_ptr(), q.ld_out = q.n;
        } else {
            const at::Tensor& o = tensor("out", a[5]);
            q.ld_out = matrix("out", o, q.m, q.n, type, k.dev);
            q.out = o.data_ptr();
        }
        check(kd_linear(&q, stream_of(k.dev)));
        if (a[5] == Py_None) return THPVariable_Wrap(std::move(fresh));
        changed(tensor("out", a[5]));
        Py_INCREF(a[5]);
        return a[5];
    });
}

Kind gated_args(PyObject* const* a, PyObject* act, kd_gated_args* q) {
    const at::Tensor &x = tensor("x", a[0]), &wg = tensor("wg", a[1]), &wu = tensor("wu", a[2]);
    const Kind k = kind_of("x", x, 2);
    if (wg.dim() != 2) refuse("wg must be a 2-D tensor");
    q->dtype = k.code, q->act = act_id(act);
    q->m = x.size(0), q->d = x.size(1), q->f = wg.size(0);
    q->x = x.data_ptr(), q->ld_x = matrix("x", x, q->m, q->d, k.type, k.dev);
    q->wg = wg.data_ptr(), q->ld_wg = matrix("wg", wg, q->f, q->d, k.type, k.dev);
    q->wu = wu.data_ptr(), q->ld_wu = matrix("wu", wu, q->f, q->d, k.type, k.dev);
    return k;
}

// gated_ffn(x, wg, wu, act, out)
PyObject* gated_ffn(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        args_of(n_args, 5);
        kd_gated_args q{};
        const Kind k = gated_args(a, a[3], &q);
        c10::cuda::OptionalCUDAGuard guard;
        if (k.dev != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)k.dev);
        if (a[4] == Py_None) {
            at::Tensor out = empty({q.m, q.f}, k.type, k.dev);
            check(kd_gated_ffn(&q, out.data_ptr(), q.f, stream_of(k.dev)));
            return THPVariable_Wrap(std::move(out));
        }
        const at::Tensor& o = tensor("out", a[4]);
        const int64_t ld = matrix("out", o, q.m, q.f, k.type, k.dev);
        check(kd_gated_ffn(&q, o.data_ptr(), ld, stream_of(k.dev)));
        changed(o);
        Py_INCREF(a[4]);
        return a[4];
    });
}

// gated_ffn_backward(x, wg, wu, dh, act)
PyObject* gated_ffn_backward(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        args_of(n_args, 5);
        kd_gated_args q{};
        const Kind k = gated_args(a, a[4], &q);
        const at::Tensor& dh = tensor("dh", a[3]);
        const int64_t ld = matrix("dh", dh, q.m, q.f, k.type, k.dev);
        c10::cuda::OptionalCUDAGuard guard;
        if (k.dev != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)k.dev);
        at::Tensor dx = empty({q.m, q.d}, k.type, k.dev), dwg = empty({q.f, q.d}, k.type, k.dev), dwu = empty({q.f, q.d}, k.type, k.dev);
        if (q.m == 0 || q.f == 0) {  // sums over nothing
            dx.zero_(), dwg.zero_(), dwu.zero_();
        } else {
            const size_t size = kd_gated_ffn_backward_workspace(q.m, q.f);
            at::Tensor ws = empty({(int64_t)size}, at::kByte, k.dev);  // goes back to the allocator in stream order
            check(kd_gated_ffn_backward(&q, dh.data_ptr(), ld, dx.data_ptr(), q.d, dwg.data_ptr(), q.d, dwu.data_ptr(), q.d,
                                        ws.data_ptr(), size, stream_of(k.dev)));
        }
        PyObject* t = PyTuple_New(3);
        if (!t) throw Refused();
        PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(dx)));
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(dwg)));
        PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(std::move(dwu)));
        return t;
    });
}

// prompt_attention(q, k, v, kv_len, scale, out)
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded([&]() -> PyObject* {
        args_of(n_args, 6);
        const at::Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]), &v = tensor("v", a[2]);
        const Kind kind = kind_of("q", q, 3);
        kd_attention_args p{};
        p.dtype = kind.code;
        p.n = q.size(0);
        p.kv_len = PyLong_AsLongLong(a[3]);
        if (p.kv_len == -1 && PyErr_Occurred()) throw Refused();
        if (p.kv_len < 0) refuse("kv_len must not be negative");
        if (p.kv_len > INT32_MAX) refuse("kv_len is out of range");
        const int64_t hd = q.size(2);
        for (int i = 0; i < 2; ++i) {
            const at::Tensor& t = i ? v : k;
            const char* name = i ? "v" : "k";
            same(name, t, kind.type, kind.dev);
            if (t.dim() != 3 || t.size(2) != hd || t.size(0) != k.size(0) || t.size(1) < p.kv_len + p.n)
                refuse("%s has shape %s: need (%lld, >= %lld, %lld)", name, shape_of(t).c_str(), (long long)k.size(0),
                       (long long)(p.kv_len + p.n), (long long)hd);
            if (hd > 1 && t.stride(2) != 1) refuse("%s: the last dimension must be contiguous", name);
        }
        if (hd > 1 && q.stride(2) != 1) refuse("q: the last dimension must be contiguous");
        if (q.size(1) > INT32_MAX || k.size(0) > INT32_MAX || hd > INT32_MAX) refuse("too many heads");
        p.n_heads = (int32_t)q.size(1), p.n_kv_heads = (int32_t)k.size(0), p.head_dim = (int32_t)hd;
        p.scale = a[4] == Py_None ? (hd > 0 ? 1.f / std::sqrt((float)hd) : 0.f) : (float)PyFloat_AsDouble(a[4]);
        if (PyErr_Occurred()) throw Refused();
        p.q = q.data_ptr(), p.q_token = q.stride(0), p.q_head = q.stride(1);
        p.k = k.data_ptr(), p.k_pos = k.stride(1), p.k_head = k.stride(0);
        p.v = v.data_ptr(), p.v_pos = v.stride(1), p.v_head = v.stride(0);
        c10::cuda::OptionalCUDAGuard guard;
        if (kind.dev != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)kind.dev);
        at::Tensor out;
        if (a[5] == Py_None) {
            out = empty({p.n, q.size(1), hd}, kind.type, kind.dev);
        } else {
            out = tensor("out", a[5]);
            same("out", out, kind.type, kind.dev);
            if (out.sizes() != q.sizes() || (hd > 1 && out.stride(2) != 1)) refuse("out must have q's shape, the last dimension contiguous");
        }
        p.out = out.data_ptr(), p.out_token = out.stride(0), p.out_head = out.stride(1);
        at::Tensor ws;
        p.workspace_bytes = kd_prompt_attention_workspace(&p);
        if (p.workspace_bytes) {
            ws = empty({(int64_t)p.workspace_bytes}, at::kByte, kind.dev);
            p.workspace = ws.data_ptr();
        }
        check(kd_prompt_attention(&p, stream_of(kind.dev)));
        if (a[5] == Py_None) return THPVariable_Wrap(std::move(out));
        changed(out);
        Py_INCREF(a[5]);
        return a[5];
    });
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, nullptr},
    {"gated_ffn", (PyCFunction)(void (*)(void))gated_ffn, METH_FASTCALL, nullptr},
    {"gated_ffn_backward", (PyCFunction)(void (*)(void))gated_ffn_backward, METH_FASTCALL, nullptr},
    {"prompt_attention", (PyCFunction)(void (*)(void))prompt_attention, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kd_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kd_torch(void) { return PyModule_Create(&module); }
