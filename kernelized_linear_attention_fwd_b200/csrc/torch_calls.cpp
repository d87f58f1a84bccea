// Short cut of the Python binding for the calls whose kernels take a few
// microseconds: checks, output allocation and the C call in one step instead of
// some forty Python operations (host time of a decode step's head norm: 20 us in
// Python, 8 here; of the gradient of a small cross attention: 26 and 14).
//
// Every function takes the binding's arguments by position and either makes the
// call and returns its outputs, or returns the library's status (an int) when the
// library refused, or NotImplemented when the arguments are not the plain case
// (exact torch tensors, CUDA, of the current device, expected shapes and types):
// the Python code then goes through them and raises the error with its message.
// Holds the addresses of the C functions and nothing else.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kata.h"

namespace {

decltype(&kata_qk_norm_rotate) g_norm;
decltype(&kata_qk_norm_rotate_backward) g_norm_bwd;
decltype(&kata_qk_norm_rotate_backward_workspace_bytes) g_norm_ws;
decltype(&kata_cross_forward) g_fwd;
decltype(&kata_cross_forward_workspace_bytes) g_fwd_ws;
decltype(&kata_cross_backward) g_bwd;
decltype(&kata_cross_backward_workspace_bytes) g_bwd_ws;

using Sizes = at::IntArrayRef;

// Not the plain case: the Python code takes over.
struct Other {};

// The arguments of one call.
struct Args {
    PyObject *const *a;
    Py_ssize_t n, i = 0;
    at::Device device = at::Device(at::kCPU);

    PyObject *next() {
        if (i >= n) throw Other{};
        return a[i++];
    }
    const at::Tensor &tensor() {
        PyObject *o = next();
        if (!THPVariable_CheckExact(o)) throw Other{};
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.layout() != at::kStrided) throw Other{};
        return t;
    }
    // the first tensor, which names the device: the current one
    const at::Tensor &first() {
        const at::Tensor &t = tensor();
        device = t.device();
        if (device.index() != c10::cuda::current_device()) throw Other{};
        return t;
    }
    // a tensor of this device, or nullptr for None
    const at::Tensor *optional() {
        if (i < n && a[i] == Py_None) {
            ++i;
            return nullptr;
        }
        const at::Tensor &t = tensor();
        if (t.device() != device) throw Other{};
        return &t;
    }
    // dense, of these sizes and this type
    const at::Tensor *dense(Sizes sizes, at::ScalarType type) {
        const at::Tensor *t = optional();
        if (t && (t->sizes() != sizes || t->scalar_type() != type || !t->is_contiguous())) throw Other{};
        return t;
    }
    const at::Tensor &required(Sizes sizes, at::ScalarType type) {
        const at::Tensor *t = dense(sizes, type);
        if (!t) throw Other{};
        return *t;
    }
    double number() {
        const double x = PyFloat_AsDouble(next());
        if (x == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            throw Other{};
        }
        return x;
    }
    bool truth() {
        const int x = PyObject_IsTrue(next());
        if (x < 0) {
            PyErr_Clear();
            throw Other{};
        }
        return x != 0;
    }
    at::Tensor make(const at::Tensor *given, Sizes sizes, at::ScalarType type) const {
        if (given) return *given;
        return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
    }
    // (tensor kept alive, address, bytes) of a workspace
    at::Tensor workspace(const at::Tensor *given, size_t need, void *&p, size_t &bytes) const {
        at::Tensor t;
        if (given) {
            if (!given->is_contiguous()) throw Other{};
            t = *given;
        } else if (need > 0) {
            t = make(nullptr, {(int64_t)need}, at::kByte);
        }
        p = t.defined() ? t.data_ptr() : nullptr;
        bytes = t.defined() ? t.nbytes() : 0;
        return t;
    }
    kata_stream_t stream() const {
        return reinterpret_cast<kata_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
    }
};

kata_dtype code(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return KATA_BF16;
    if (t.scalar_type() == at::kFloat) return KATA_F32;
    throw Other{};
}
int narrow(int64_t x) {
    if (x < 0 || x > 0x7fffffff) throw Other{};
    return (int)x;
}
template <typename P>
P *ptr(const at::Tensor *t) {
    return t ? static_cast<P *>(t->data_ptr()) : nullptr;
}
void *ptr(const at::Tensor &t) { return t.data_ptr(); }

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}
template <size_t N>
PyObject *wrap_all(const std::array<at::Tensor, N> &ts) {
    PyObject *r = PyTuple_New(N);
    if (!r) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject *o = wrap(ts[i]);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i, o);
    }
    return r;
}

// Runs `f(args)`; anything that goes wrong before the C call hands over to Python,
// which meets it again and reports it.
template <typename F>
PyObject *guarded(PyObject *const *a, Py_ssize_t n, F f) {
    try {
        at::AutoDispatchBelowADInplaceOrView below;
        Args args{a, n};
        return f(args);
    } catch (const Other &) {
    } catch (const std::exception &) {
    }
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

// Queries, keys and what both directions share of them.
struct Norm {
    at::Tensor q;
    const at::Tensor *k, *qw, *kw, *inv, *pos;
    int B, T, Hq, Hk = 0, d, n_rot = 0;
    int64_t qs[3], ks[3] = {0, 0, 0}, pos_stride = 0;
    kata_dtype type;
    float eps;
    int inter;

    static void strides(const at::Tensor &t, int64_t (&s)[3]) {
        if (t.dim() != 4 || (t.size(3) > 1 && t.stride(3) != 1)) throw Other{};
        for (int i = 0; i < 3; ++i) s[i] = t.stride(i);
    }
    explicit Norm(Args &a) {
        q = a.first();
        strides(q, qs);
        B = narrow(q.size(0));
        T = narrow(q.size(1));
        Hq = narrow(q.size(2));
        d = narrow(q.size(3));
        type = code(q);
        k = a.optional();
        if (k) {
            strides(*k, ks);
            if (k->size(0) != B || k->size(1) != T || k->size(3) != d || k->scalar_type() != q.scalar_type())
                throw Other{};
            Hk = narrow(k->size(2));
        }
        qw = a.dense({d}, at::kFloat);
        kw = a.dense({d}, at::kFloat);
        if (kw && !k) throw Other{};
        inv = a.optional();
        if (inv) {
            if (inv->dim() != 1 || inv->scalar_type() != at::kFloat || !inv->is_contiguous()) throw Other{};
            n_rot = narrow(inv->size(0));
        }
        pos = a.optional();
        if (pos) {
            const bool both = pos->dim() == 2;
            if (pos->scalar_type() != at::kLong || (!both && pos->dim() != 1) || pos->size(-1) != T ||
                (both && pos->size(0) != B) || (T > 1 && pos->stride(-1) != 1))
                throw Other{};
            pos_stride = both && B > 1 ? pos->stride(0) : 0;
        }
        eps = (float)a.number();
        inter = a.truth();
    }
    const float *inv_freq() const { return n_rot ? ptr<float>(inv) : nullptr; }
};

PyObject *qk_norm_rotate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, [](Args &a) -> PyObject * {
        const Norm x(a);
        const int64_t qo[4] = {x.B, x.Hq, x.T, x.d}, ko[4] = {x.B, x.Hk, x.T, x.d};
        const at::Tensor *gq = a.dense(qo, x.q.scalar_type()), *gk = a.dense(ko, x.q.scalar_type());
        if (gk && !x.k) throw Other{};
        std::array<at::Tensor, 2> o;
        o[0] = a.make(gq, qo, x.q.scalar_type());
        if (x.k) o[1] = a.make(gk, ko, x.q.scalar_type());
        const kata_status st =
            g_norm(ptr(x.q), ptr<void>(x.k), ptr(o[0]), x.k ? ptr(o[1]) : nullptr, ptr<float>(x.qw), ptr<float>(x.kw),
                   x.inv_freq(), ptr<int64_t>(x.pos), x.B, x.T, x.Hq, x.Hk, x.d, x.n_rot, x.qs, x.k ? x.ks : nullptr,
                   x.pos_stride, x.eps, x.inter, x.type, a.stream());
        return st == KATA_OK ? wrap_all(o) : PyLong_FromLong(st);
    });
}

PyObject *qk_norm_rotate_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, [](Args &a) -> PyObject * {
        const Norm x(a);
        const at::ScalarType ty = x.q.scalar_type();
        const int64_t qo[4] = {x.B, x.Hq, x.T, x.d}, ko[4] = {x.B, x.Hk, x.T, x.d};
        const at::Tensor &gq = a.required(qo, ty);
        const at::Tensor *gk = a.dense(ko, ty);
        if (!gk != !x.k) throw Other{};
        const int64_t qi[4] = {x.B, x.T, x.Hq, x.d}, ki[4] = {x.B, x.T, x.Hk, x.d};
        std::array<at::Tensor, 4> o;  // dq, dk, dq_weight, dk_weight
        int64_t s[2][3];
        for (int m = 0; m < 2; ++m) {
            const at::Tensor *t = a.optional();
            if (m == 1 && !x.k) {
                if (t) throw Other{};
                continue;
            }
            const Sizes want(m ? ki : qi, 4);
            if (t && (t->sizes() != want || t->scalar_type() != ty)) throw Other{};
            o[m] = a.make(t, want, ty);
            Norm::strides(o[m], s[m]);
        }
        for (int m = 0; m < 2; ++m) {
            const at::Tensor *t = a.dense({x.d}, at::kFloat);
            if (m == 1 && !x.k) {
                if (t) throw Other{};
                continue;
            }
            o[2 + m] = a.make(t, {x.d}, at::kFloat);
        }
        void *ws;
        size_t bytes;
        const at::Tensor keep = a.workspace(a.optional(), g_norm_ws(x.B, x.T, x.Hq, x.Hk, x.d), ws, bytes);
        const kata_status st = g_norm_bwd(
            ptr(gq), ptr<void>(gk), ptr(x.q), ptr<void>(x.k), ptr<float>(x.qw), ptr<float>(x.kw), x.inv_freq(),
            ptr<int64_t>(x.pos), ptr(o[0]), x.k ? ptr(o[1]) : nullptr, static_cast<float *>(ptr(o[2])),
            x.k ? static_cast<float *>(ptr(o[3])) : nullptr, x.B, x.T, x.Hq, x.Hk, x.d, x.n_rot, x.qs,
            x.k ? x.ks : nullptr, s[0], x.k ? s[1] : nullptr, x.pos_stride, x.eps, x.inter, x.type, ws, bytes,
            a.stream());
        return st == KATA_OK ? wrap_all(o) : PyLong_FromLong(st);
    });
}

struct Cross {
    at::Tensor q, k, v;
    const at::Tensor *len;
    int B, H, Hkv, Tq, Tk, d;
    kata_dtype type;

    explicit Cross(Args &a) {
        q = a.first();
        const at::Tensor *kk = a.optional();
        if (!kk || q.dim() != 4 || kk->dim() != 4 || !q.is_contiguous()) throw Other{};
        k = *kk;
        B = narrow(q.size(0));
        H = narrow(q.size(1));
        Tq = narrow(q.size(2));
        d = narrow(q.size(3));
        Hkv = narrow(k.size(1));
        Tk = narrow(k.size(2));
        type = code(q);
        const int64_t want[4] = {B, Hkv, Tk, d};
        if (k.sizes() != Sizes(want, 4) || k.scalar_type() != q.scalar_type() || !k.is_contiguous()) throw Other{};
        v = a.required(want, q.scalar_type());
        len = a.dense({B}, at::kInt);
    }
};

PyObject *cross_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, [](Args &a) -> PyObject * {
        const Cross x(a);
        const at::Tensor *out = a.dense(x.q.sizes(), x.q.scalar_type()), *y = a.dense(x.q.sizes(), at::kFloat),
                         *den = a.dense({x.B, x.H, x.Tq}, at::kFloat);
        const at::Tensor o = a.make(out, x.q.sizes(), x.q.scalar_type());
        void *ws;
        size_t bytes;
        const at::Tensor keep =
            a.workspace(a.optional(), g_fwd_ws(x.B, x.H, x.Hkv, x.Tq, x.Tk, x.d, x.type), ws, bytes);
        const kata_status st =
            g_fwd(ptr(x.q), ptr(x.k), ptr(x.v), ptr<int32_t>(x.len), ptr(o), x.B, x.H, x.Hkv, x.Tq, x.Tk, x.d, x.type,
                  ptr<float>(y), ptr<float>(den), ws, bytes, a.stream());
        return st == KATA_OK ? wrap(o) : PyLong_FromLong(st);
    });
}

PyObject *cross_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(a, n, [](Args &a) -> PyObject * {
        const Cross x(a);
        const at::ScalarType ty = x.q.scalar_type();
        const at::Tensor &g = a.required(x.q.sizes(), ty), &y = a.required(x.q.sizes(), at::kFloat),
                         &den = a.required({x.B, x.H, x.Tq}, at::kFloat);
        std::array<at::Tensor, 3> o;
        for (int m = 0; m < 3; ++m) {
            const Sizes want = m == 0 ? x.q.sizes() : x.k.sizes();
            o[m] = a.make(a.dense(want, ty), want, ty);
        }
        void *ws;
        size_t bytes;
        const at::Tensor keep =
            a.workspace(a.optional(), g_bwd_ws(x.B, x.H, x.Hkv, x.Tq, x.Tk, x.d, x.type), ws, bytes);
        const kata_status st =
            g_bwd(ptr(g), ptr(x.q), ptr(x.k), ptr(x.v), static_cast<float *>(ptr(y)), static_cast<float *>(ptr(den)),
                  ptr<int32_t>(x.len), ptr(o[0]), ptr(o[1]), ptr(o[2]), x.B, x.H, x.Hkv, x.Tq, x.Tk, x.d, x.type, ws,
                  bytes, a.stream());
        return st == KATA_OK ? wrap_all(o) : PyLong_FromLong(st);
    });
}

// bind(addresses): of the C functions, in the order of the globals above.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    void *p[7];
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes 7 addresses");
        return nullptr;
    }
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    g_norm = reinterpret_cast<decltype(g_norm)>(p[0]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[1]);
    g_norm_ws = reinterpret_cast<decltype(g_norm_ws)>(p[2]);
    g_fwd = reinterpret_cast<decltype(g_fwd)>(p[3]);
    g_fwd_ws = reinterpret_cast<decltype(g_fwd_ws)>(p[4]);
    g_bwd = reinterpret_cast<decltype(g_bwd)>(p[5]);
    g_bwd_ws = reinterpret_cast<decltype(g_bwd_ws)>(p[6]);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"),
                           method<qk_norm_rotate>("qk_norm_rotate"),
                           method<qk_norm_rotate_backward>("qk_norm_rotate_backward"),
                           method<cross_forward>("cross_forward"),
                           method<cross_backward>("cross_backward"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&g_module); }
