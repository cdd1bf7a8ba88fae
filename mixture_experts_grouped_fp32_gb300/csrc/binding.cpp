// binding.cpp — the usual calls of the training operators without Python's share of their cost: checks of
// the tensors, output allocation and the C call in one go.
//
// Every function takes what the Python function of the same name takes and returns its result; None if
// anything is out of the ordinary (another type, shape, device or layout), which the Python function then
// reports; or an int, the C call's error code.  It adds no behaviour of its own: without this module the
// Python functions do the same through ctypes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "../../include/moe.h"

namespace {

#define MOE_FAST_CALLS(X)                                                                                   \
    X(moe_swiglu) X(moe_swiglu_backward) X(moe_block_norm) X(moe_block_norm_backward)                       \
    X(moe_block_norm_backward_workspace_size) X(moe_grouped_mm) X(moe_grouped_mm_wgrad)                     \
    X(moe_grouped_mm_workspace_size) X(moe_adamw_step)
// Calls that a library may lack: their functions here then leave the work to the Python ones.
#define MOE_FAST_MORE_CALLS(X)                                                                              \
    X(moe_route_scores) X(moe_route_scores_backward) X(moe_layer_norm) X(moe_layer_norm_backward)           \
    X(moe_layer_norm_backward_workspace_size) X(moe_dropout) X(moe_embed) X(moe_embed_backward)             \
    X(moe_embed_backward_workspace_size)
struct Lib {
#define X(name) decltype(&::name) name = nullptr;
    MOE_FAST_CALLS(X)
    MOE_FAST_MORE_CALLS(X)
#undef X
} lib;

using at::ScalarType;
constexpr ScalarType BF16 = ScalarType::BFloat16, F32 = ScalarType::Float, I32 = ScalarType::Int;

// The tensor behind an argument, or nullptr.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Operands of one call: `ok` stays true while all are contiguous CUDA tensors of the wanted type and shape, on the
// current device (where the call launches).
struct Args {
    bool ok = true;
    int current = -1;
    bool here(const at::Tensor& t) {  // (asking for the current device costs 0.15 us, and one device needs none of it)
        static const bool several = c10::cuda::device_count() > 1;
        if (several && current < 0) current = c10::cuda::current_device();
        return !several || t.get_device() == current;
    }
    const at::Tensor* need(PyObject* o, int dims) {
        const at::Tensor* t = tensor(o);
        if (!t || t->dim() != dims) ok = false;
        return ok ? t : nullptr;
    }
    void* plain(const at::Tensor& t, ScalarType type) {
        if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous() || !here(t)) ok = false;
        return ok ? t.data_ptr() : nullptr;
    }
    void* at(PyObject* o, ScalarType type, at::IntArrayRef shape, bool optional = false) {
        if (!ok || (optional && o == Py_None)) return nullptr;
        const at::Tensor* t = tensor(o);
        if (!t || t->sizes() != shape) {
            ok = false;
            return nullptr;
        }
        return plain(*t, type);
    }
    void* opt(PyObject* o, ScalarType type, at::IntArrayRef shape) { return at(o, type, shape, true); }
};

at::Tensor make(at::IntArrayRef shape, ScalarType type, const at::Tensor& like) {
    return at::Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject* wrap(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject* code(int rc) { return PyLong_FromLong(rc); }
moe_stream_t stream() { return c10::cuda::getCurrentCUDAStream().stream(); }
bool fits(int64_t v) { return v >= 0 && v < (1ll << 31); }

// Runs a function's body; a C++ exception becomes the Python one that torch's own functions raise for it (an
// allocation that failed: torch.OutOfMemoryError).
template <typename F>
PyObject* guarded(F body) {
    HANDLE_TH_ERRORS
    return body();
    END_HANDLE_TH_ERRORS
}

// A C call without the interpreter lock, as ctypes makes it: a launch waits where the launch queue is full, perhaps
// for a host function on the stream that needs the lock.
template <typename F>
int unlocked(F call) {
    struct Lock {
        PyThreadState* state = PyEval_SaveThread();
        ~Lock() { PyEval_RestoreThread(state); }
    } released;
    return call();
}

// Tells autograd that a tensor of the caller's has been written to.
void touch(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// swiglu(gu, w)
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* gu = n == 2 ? c.need(a[0], 2) : nullptr;
        if (!gu || gu->size(1) % 2 || !fits(gu->size(0)) || !fits(gu->size(1))) Py_RETURN_NONE;
        const int64_t M = gu->size(0), f = gu->size(1) / 2;
        const void* pg = c.plain(*gu, BF16);
        const void* pw = c.opt(a[1], F32, {M});
        if (!c.ok) Py_RETURN_NONE;
        at::Tensor h = make({M, f}, BF16, *gu);
        const int rc = unlocked([&] {
            return lib.moe_swiglu(pg, static_cast<const float*>(pw), M, f, ptr(h), stream());
        });
        return rc ? code(rc) : wrap(h);
    });
}

// swiglu_backward(gu, dh, w, want_h) -> (dgu, dw, h)
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* gu = n == 4 ? c.need(a[0], 2) : nullptr;
        if (!gu || gu->size(1) % 2 || !fits(gu->size(0)) || !fits(gu->size(1))) Py_RETURN_NONE;
        const int64_t M = gu->size(0), f = gu->size(1) / 2;
        const void* pg = c.plain(*gu, BF16);
        const void* pd = c.at(a[1], BF16, {M, f});
        const void* pw = c.opt(a[2], F32, {M});
        if (!c.ok) Py_RETURN_NONE;
        at::Tensor dgu = make({M, 2 * f}, BF16, *gu), dw, h;
        if (a[2] != Py_None) dw = make({M}, F32, *gu);
        if (PyObject_IsTrue(a[3])) h = make({M, f}, BF16, *gu);
        const int rc = unlocked([&] {
            return lib.moe_swiglu_backward(pg, pd, static_cast<const float*>(pw), M, f, ptr(dgu),
                                           static_cast<float*>(ptr(dw)), ptr(h), stream());
        });
        return rc ? code(rc) : Py_BuildValue("(NNN)", wrap(dgu), wrap(dw), wrap(h));
    });
}

// The inputs that both norm calls take: a[0] x, a[i..] w_pre, h, w_post, gate, token_gate, res_scale.
struct Norm {
    Args c;
    const at::Tensor* x = nullptr;
    int64_t T = 0, d = 0;
    ScalarType type = F32;
    const void *px = nullptr, *h = nullptr;
    const float *w_pre = nullptr, *w_post = nullptr, *gate = nullptr, *tgate = nullptr, *res = nullptr;
    bool has_h = false, has_pre = false;

    bool read(PyObject* xo, PyObject* const* a) {
        x = c.need(xo, 2);
        if (!x || (x->scalar_type() != BF16 && x->scalar_type() != F32) || !fits(x->size(0)) || !fits(x->size(1)))
            return false;
        T = x->size(0), d = x->size(1), type = x->scalar_type();
        px = c.plain(*x, type);
        auto vec = [&](PyObject* o, int64_t size) { return static_cast<const float*>(c.opt(o, F32, {size})); };
        has_pre = a[0] != Py_None, has_h = a[1] != Py_None;
        w_pre = vec(a[0], d);
        h = c.opt(a[1], BF16, {T, d});
        w_post = vec(a[2], d), gate = vec(a[3], d), tgate = vec(a[4], T), res = vec(a[5], d);
        return c.ok;
    }
};

// block_norm(x, w_pre, h, w_post, gate, token_gate, res_scale, eps) -> (y, n)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Norm v;
        if (n != 8 || !v.read(a[0], a + 1)) Py_RETURN_NONE;
        const double eps = PyFloat_AsDouble(a[7]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        at::Tensor y, out;
        if (v.has_h) y = make({v.T, v.d}, v.type, *v.x);
        if (v.has_pre) out = make({v.T, v.d}, BF16, *v.x);
        const int rc = unlocked([&] {
            return lib.moe_block_norm(v.px, v.type == F32, v.h, v.w_pre, v.w_post, v.gate, v.tgate, v.res, v.T,
                                      v.d, static_cast<float>(eps), ptr(y), ptr(out), stream());
        });
        return rc ? code(rc) : Py_BuildValue("(NN)", wrap(y), wrap(out));
    });
}

// block_norm_backward(x, dy, dn, w_pre, h, w_post, gate, token_gate, res_scale, eps)
//   -> gradients of (x, h, w_pre, w_post, gate, token_gate, res_scale)
PyObject* block_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Norm v;
        if (n != 10 || !v.read(a[0], a + 3)) Py_RETURN_NONE;
        const void* dy = v.c.opt(a[1], v.type, {v.T, v.d});
        const void* dn = v.c.opt(a[2], BF16, {v.T, v.d});
        if (!v.c.ok) Py_RETURN_NONE;
        const double eps = PyFloat_AsDouble(a[9]);
        if (eps == -1.0 && PyErr_Occurred()) return nullptr;
        const size_t need = lib.moe_block_norm_backward_workspace_size(v.T, v.d);
        at::Tensor ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, *v.x);
        at::Tensor g[7];
        g[0] = make({v.T, v.d}, v.type, *v.x);
        if (v.has_h) g[1] = make({v.T, v.d}, BF16, *v.x);
        if (v.has_pre && a[2] != Py_None) g[2] = make({v.d}, F32, *v.x);
        for (int k = 0; k < 4; ++k)  // w_post, gate, token_gate, res_scale
            if (a[5 + k] != Py_None) g[3 + k] = make({k == 2 ? v.T : v.d}, F32, *v.x);
        auto f = [&](int k) { return static_cast<float*>(ptr(g[k])); };
        const int rc = unlocked([&] {
            return lib.moe_block_norm_backward(v.px, v.type == F32, v.h, dy, dn, v.w_pre, v.w_post, v.gate, v.tgate,
                                               v.res, v.T, v.d, static_cast<float>(eps), ptr(g[0]), ptr(g[1]), f(2),
                                               f(3), f(4), f(5), f(6), ptr(ws), need, stream());
        });
        return rc ? code(rc)
                  : Py_BuildValue("(NNNNNNN)", wrap(g[0]), wrap(g[1]), wrap(g[2]), wrap(g[3]), wrap(g[4]), wrap(g[5]),
                                  wrap(g[6]));
    });
}

// grouped_mm(a, b, offsets, transpose_b, fp32, status)
PyObject* grouped_mm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* x = n == 6 ? c.need(a[0], 2) : nullptr;
        const at::Tensor* w = x ? c.need(a[1], 3) : nullptr;
        if (!w) Py_RETURN_NONE;
        const bool trans = PyObject_IsTrue(a[3]), f32 = PyObject_IsTrue(a[4]);
        const int64_t M = x->size(0), K = x->size(1), E = w->size(0), N = w->size(trans ? 1 : 2);
        if (!fits(M) || !fits(K) || !fits(E) || !fits(N) || w->size(trans ? 2 : 1) != K) Py_RETURN_NONE;
        const void *pa = c.plain(*x, BF16), *pb = c.plain(*w, BF16), *po = c.at(a[2], I32, {E + 1});
        void* st = c.opt(a[5], I32, {1});
        if (!c.ok) Py_RETURN_NONE;
        const size_t need = lib.moe_grouped_mm_workspace_size(trans ? 1 : 0, M, K, N, E);
        at::Tensor ws, out = make({M, N}, f32 ? F32 : BF16, *x);
        if (need) ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, *x);
        const int rc = unlocked([&] {
            return lib.moe_grouped_mm(pa, pb, static_cast<const int32_t*>(po), M, K, N, E, trans, ptr(out), f32,
                                      ptr(ws), need, static_cast<int32_t*>(st), stream());
        });
        return rc ? code(rc) : wrap(out);
    });
}

// grouped_mm_wgrad(a, g, offsets, out or None, fp32, accumulate, status)
PyObject* grouped_mm_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* x = n == 7 ? c.need(a[0], 2) : nullptr;
        const at::Tensor* g = x ? c.need(a[1], 2) : nullptr;
        const at::Tensor* o = g ? c.need(a[2], 1) : nullptr;
        if (!o) Py_RETURN_NONE;
        const bool f32 = PyObject_IsTrue(a[4]), acc = PyObject_IsTrue(a[5]);
        const int64_t M = x->size(0), K = x->size(1), N = g->size(1), E = o->size(0) - 1;
        if (!fits(M) || !fits(K) || !fits(E) || !fits(N) || g->size(0) != M || E < 1) Py_RETURN_NONE;
        const void *pa = c.plain(*x, BF16), *pg = c.plain(*g, BF16), *po = c.plain(*o, I32);
        c.opt(a[3], f32 ? F32 : BF16, {E, K, N});
        void* st = c.opt(a[6], I32, {1});
        if (!c.ok || (acc && a[3] == Py_None)) Py_RETURN_NONE;
        const size_t need = lib.moe_grouped_mm_workspace_size(2, M, K, N, E);
        at::Tensor ws, out = a[3] == Py_None ? make({E, K, N}, f32 ? F32 : BF16, *x) : *tensor(a[3]);
        if (need) ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, *x);
        const int rc = unlocked([&] {
            return lib.moe_grouped_mm_wgrad(pa, pg, static_cast<const int32_t*>(po), M, K, N, E, ptr(out), f32, acc,
                                            ptr(ws), need, static_cast<int32_t*>(st), stream());
        });
        if (rc) return code(rc);
        if (a[3] == Py_None) return wrap(out);
        touch(out);
        Py_INCREF(a[3]);
        return a[3];
    });
}

// adamw_step(params, grads, m, v, m_scales, v_scales, copies, lr, beta1, beta2, eps, weight_decay, step)
//   -> 0, an error code, or None.  Lists or tuples of tensors.
PyObject* adamw_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 13) Py_RETURN_NONE;
        for (int l = 0; l < 7; ++l)
            if (!(PyList_Check(a[l]) || PyTuple_Check(a[l]) || (l > 3 && a[l] == Py_None))) Py_RETURN_NONE;
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
        if (count == 0 || count > (1 << 20)) Py_RETURN_NONE;
        for (int l = 1; l < 7; ++l)
            if (a[l] != Py_None && PySequence_Fast_GET_SIZE(a[l]) != count) Py_RETURN_NONE;
        const at::Tensor* first[3] = {tensor(PySequence_Fast_GET_ITEM(a[0], 0)), tensor(PySequence_Fast_GET_ITEM(a[1], 0)),
                                      tensor(PySequence_Fast_GET_ITEM(a[2], 0))};
        if (!first[0] || !first[1] || !first[2]) Py_RETURN_NONE;
        const ScalarType pt = first[0]->scalar_type(), gt = first[1]->scalar_type(), st = first[2]->scalar_type();
        const bool eight = st == ScalarType::Float8_e4m3fn;
        if ((pt != F32 && pt != BF16) || (gt != F32 && gt != BF16) || (st != F32 && !eight)) Py_RETURN_NONE;
        if (eight != (a[4] != Py_None) || eight != (a[5] != Py_None)) Py_RETURN_NONE;
        const ScalarType types[7] = {pt, gt, st, st, F32, F32, BF16};
        static thread_local std::vector<moe_adamw_tensor> table;
        table.assign(count, moe_adamw_tensor{});
        Args c;
        for (int l = 0; l < 7; ++l) {
            if (a[l] == Py_None) continue;
            PyObject** items = PySequence_Fast_ITEMS(a[l]);
            for (Py_ssize_t i = 0; i < count; ++i) {
                const at::Tensor* t = tensor(items[i]);
                if (!t) Py_RETURN_NONE;
                moe_adamw_tensor& e = table[i];
                if (l == 0) e.n = t->numel();
                const int64_t want = l == 4 || l == 5 ? (e.n + 255) / 256 : e.n;
                void* p = c.plain(*t, types[l]);
                if (!c.ok || t->numel() != want) Py_RETURN_NONE;
                if (l == 0 || l == 6) touch(*t);
                switch (l) {
                    case 0: e.param = p; break;
                    case 1: e.grad = p; break;
                    case 2: e.m = p; break;
                    case 3: e.v = p; break;
                    case 4: e.m_scale = static_cast<float*>(p); break;
                    case 5: e.v_scale = static_cast<float*>(p); break;
                    default: e.copy = p;
                }
            }
        }
        double h[5];
        for (int k = 0; k < 5; ++k) {
            h[k] = PyFloat_AsDouble(a[7 + k]);
            if (h[k] == -1.0 && PyErr_Occurred()) return nullptr;
        }
        const long step = PyLong_AsLong(a[12]);
        if (step == -1 && PyErr_Occurred()) return nullptr;
        if (step < 1 || step > 0x7fffffff) Py_RETURN_NONE;
        const int rc = unlocked([&] {
            return lib.moe_adamw_step(table.data(), static_cast<int>(count), pt == BF16, gt == BF16, eight ? 8 : 32, h[0],
                                      h[1], h[2], h[3], h[4], static_cast<int>(step), nullptr, nullptr, stream());
        });
        return code(rc);
    });
}

// A Python integer or number that fits, else false (and no error is left behind: the Python function reports it).
template <typename V, typename F>
bool number(F convert, PyObject* o, V* out) {
    const auto v = convert(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    *out = static_cast<V>(v);
    return static_cast<decltype(v)>(*out) == v || v != v;
}
bool integer(PyObject* o, int* out) { return PyLong_Check(o) && number(PyLong_AsLong, o, out); }
bool real(PyObject* o, double* out) { return number(PyFloat_AsDouble, o, out); }
bool real(PyObject* o, float* out) {
    double v;
    if (!real(o, &v)) return false;
    *out = static_cast<float>(v);
    return true;
}
bool one_of(ScalarType t) { return t == BF16 || t == F32; }

// Whether an object is true; false is returned for one that has no answer (the Python function reports it).
bool truth(PyObject* o, bool* out) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) PyErr_Clear();
    *out = v > 0;
    return v >= 0;
}

// "softmax" 0, "sigmoid" 1, anything else -1.
int scoring_of(PyObject* o) {
    if (!PyUnicode_Check(o)) return -1;
    return PyUnicode_CompareWithASCIIString(o, "softmax") == 0 ? 0 : PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0 ? 1 : -1;
}

// route_scores(logits, top_k, scoring, bias, n_group, topk_group, renormalize, scale, want_scores) -> (idx, w, scores)
PyObject* route_scores(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* l = n == 9 && lib.moe_route_scores ? c.need(a[0], 2) : nullptr;
        if (!l || !one_of(l->scalar_type()) || !fits(l->size(0)) || !fits(l->size(1))) Py_RETURN_NONE;
        const int64_t T = l->size(0), E = l->size(1);
        int k, groups, kept;
        float scale;
        const int how = scoring_of(a[2]);
        if (how < 0 || !integer(a[1], &k) || !integer(a[4], &groups) || !integer(a[5], &kept) || !real(a[7], &scale) || k < 1)
            Py_RETURN_NONE;
        const void *pl = c.plain(*l, l->scalar_type()), *pb = c.opt(a[3], F32, {E});
        if (!c.ok) Py_RETURN_NONE;
        bool renorm, want;
        if (!truth(a[6], &renorm) || !truth(a[8], &want)) Py_RETURN_NONE;
        at::Tensor idx = make({T, k}, I32, *l), w = make({T, k}, F32, *l), scores;
        if (want) scores = make({T, E}, F32, *l);
        const int rc = unlocked([&] {
            return lib.moe_route_scores(pl, l->scalar_type() == BF16, static_cast<const float*>(pb), T, E, k, how, groups,
                                        kept, renorm, scale, static_cast<int32_t*>(ptr(idx)), static_cast<float*>(ptr(w)),
                                        static_cast<float*>(ptr(scores)), stream());
        });
        return rc ? code(rc) : Py_BuildValue("(NNN)", wrap(idx), wrap(w), wrap(scores));
    });
}

// route_scores_backward(logits, idx, dw, dscores, scoring, renormalize, scale)
PyObject* route_scores_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* l = n == 7 && lib.moe_route_scores_backward ? c.need(a[0], 2) : nullptr;
        if (!l || !one_of(l->scalar_type()) || !fits(l->size(0)) || !fits(l->size(1))) Py_RETURN_NONE;
        const int64_t T = l->size(0), E = l->size(1);
        float scale;
        const int how = scoring_of(a[4]);
        if (how < 0 || !real(a[6], &scale)) Py_RETURN_NONE;
        int64_t k = 1;
        const void *pl = c.plain(*l, l->scalar_type()), *pi = nullptr, *pw = nullptr;
        if (a[2] != Py_None) {
            const at::Tensor* w = c.need(a[2], 2);
            if (!w || !fits(w->size(1))) Py_RETURN_NONE;
            k = w->size(1);
            pw = c.at(a[2], F32, {T, k});
            pi = c.at(a[1], I32, {T, k});
        }
        const at::Tensor* ds = tensor(a[3]);
        const bool per_token = ds && ds->dim() == 2;
        const void* ps = per_token ? c.at(a[3], F32, {T, E}) : c.opt(a[3], F32, {E});
        if (!c.ok) Py_RETURN_NONE;
        bool renorm;
        if (!truth(a[5], &renorm)) Py_RETURN_NONE;
        at::Tensor out = make({T, E}, l->scalar_type(), *l);
        const int rc = unlocked([&] {
            return lib.moe_route_scores_backward(pl, l->scalar_type() == BF16, static_cast<const int32_t*>(pi),
                                                 static_cast<const float*>(pw), static_cast<const float*>(ps), per_token, T,
                                                 E, k, how, renorm, scale, ptr(out), stream());
        });
        return rc ? code(rc) : wrap(out);
    });
}

// p, seed, offset, offset_tensor of the calls with dropout.
struct Dropping {
    double p;
    uint64_t seed;
    int64_t offset;
    const int64_t* dev;
    bool read(Args& c, PyObject* const* a) {
        if (!real(a[0], &p) || !PyLong_Check(a[1]) || !PyLong_Check(a[2])) return false;
        if (!number(PyLong_AsUnsignedLongLong, a[1], &seed) || !number(PyLong_AsLongLong, a[2], &offset)) return false;
        dev = static_cast<const int64_t*>(c.opt(a[3], ScalarType::Long, {1}));
        return c.ok;
    }
};

// dropout(x, p, seed, offset, offset_tensor, residual)
PyObject* dropout(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* x = n == 6 && lib.moe_dropout ? tensor(a[0]) : nullptr;
        if (!x || !one_of(x->scalar_type())) Py_RETURN_NONE;
        const at::Tensor* r = a[5] == Py_None ? x : tensor(a[5]);
        if (!r || !one_of(r->scalar_type())) Py_RETURN_NONE;
        Dropping drop;
        const void *px = c.plain(*x, x->scalar_type()), *pr = c.opt(a[5], r->scalar_type(), x->sizes());
        if (!c.ok || !drop.read(c, a + 1)) Py_RETURN_NONE;
        at::Tensor out = make(x->sizes(), r->scalar_type(), *x);
        const int rc = unlocked([&] {
            return lib.moe_dropout(px, x->scalar_type() == F32, pr, r->scalar_type() == F32, x->numel(), drop.p, drop.seed,
                                   drop.offset, drop.dev, ptr(out), stream());
        });
        return rc ? code(rc) : wrap(out);
    });
}

// layer_norm(x, weight, bias, h, p, seed, offset, offset_tensor, eps) -> (y, n, stats)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* x = n == 9 && lib.moe_layer_norm ? c.need(a[0], 2) : nullptr;
        if (!x || !one_of(x->scalar_type()) || !fits(x->size(0)) || !fits(x->size(1))) Py_RETURN_NONE;
        const int64_t T = x->size(0), d = x->size(1);
        const ScalarType type = x->scalar_type();
        const void *px = c.plain(*x, type), *pw = c.opt(a[1], F32, {d}), *pb = c.opt(a[2], F32, {d}),
                   *ph = c.opt(a[3], BF16, {T, d});
        Dropping drop;
        float eps;
        if (!c.ok || !drop.read(c, a + 4) || !real(a[8], &eps)) Py_RETURN_NONE;
        at::Tensor y, out = make({T, d}, BF16, *x), stats = make({T, 2}, F32, *x);
        if (a[3] != Py_None) y = make({T, d}, type, *x);
        const int rc = unlocked([&] {
            return lib.moe_layer_norm(px, type == F32, ph, static_cast<const float*>(pw), static_cast<const float*>(pb), T, d,
                                      eps, drop.p, drop.seed, drop.offset, drop.dev, ptr(y), ptr(out),
                                      static_cast<float*>(ptr(stats)), stream());
        });
        return rc ? code(rc) : Py_BuildValue("(NNN)", wrap(y), wrap(out), wrap(stats));
    });
}

// layer_norm_backward(x, stats, dn, dy, weight, bias, want_h, p, seed, offset, offset_tensor)
//   -> gradients of (x, h, weight, bias)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* x = n == 11 && lib.moe_layer_norm_backward ? c.need(a[0], 2) : nullptr;
        if (!x || !one_of(x->scalar_type()) || !fits(x->size(0)) || !fits(x->size(1))) Py_RETURN_NONE;
        const int64_t T = x->size(0), d = x->size(1);
        const ScalarType type = x->scalar_type();
        const void *px = c.plain(*x, type), *ps = c.at(a[1], F32, {T, 2}), *pn = c.at(a[2], BF16, {T, d}),
                   *py = c.opt(a[3], type, {T, d}), *pw = c.opt(a[4], F32, {d});
        c.opt(a[5], F32, {d});
        Dropping drop;
        if (!c.ok || !drop.read(c, a + 7)) Py_RETURN_NONE;
        bool want_h;
        if (!truth(a[6], &want_h)) Py_RETURN_NONE;
        const size_t need = lib.moe_layer_norm_backward_workspace_size(T, d);
        at::Tensor ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, *x), dx = make({T, d}, type, *x), dh, dw, db;
        if (want_h) dh = make({T, d}, BF16, *x);
        if (a[4] != Py_None) dw = make({d}, F32, *x);
        if (a[5] != Py_None) db = make({d}, F32, *x);
        const int rc = unlocked([&] {
            return lib.moe_layer_norm_backward(px, type == F32, static_cast<const float*>(ps), pn, py,
                                               static_cast<const float*>(pw), T, d, drop.p, drop.seed, drop.offset, drop.dev,
                                               ptr(dx), ptr(dh), static_cast<float*>(ptr(dw)), static_cast<float*>(ptr(db)),
                                               ptr(ws), need, stream());
        });
        return rc ? code(rc) : Py_BuildValue("(NNNN)", wrap(dx), wrap(dh), wrap(dw), wrap(db));
    });
}

// The ids of the embedding calls: contiguous int32 or int64 of any shape.
const at::Tensor* ids_of(Args& c, PyObject* o, const void** p) {
    const at::Tensor* t = tensor(o);
    if (!t || (t->scalar_type() != I32 && t->scalar_type() != ScalarType::Long) || !fits(t->numel())) return nullptr;
    *p = c.plain(*t, t->scalar_type());
    return c.ok ? t : nullptr;
}

// embed(ids, table, scale, whether the result is fp32 or None for the table's type, status)
PyObject* embed(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* w = n == 5 && lib.moe_embed ? c.need(a[1], 2) : nullptr;
        const void* pi = nullptr;
        const at::Tensor* ids = w ? ids_of(c, a[0], &pi) : nullptr;
        if (!ids || !one_of(w->scalar_type()) || !fits(w->size(0)) || !fits(w->size(1))) Py_RETURN_NONE;
        if (a[3] != Py_None && !PyBool_Check(a[3])) Py_RETURN_NONE;
        float scale;
        const void* pw = c.plain(*w, w->scalar_type());
        void* st = c.opt(a[4], I32, {1});
        if (!c.ok || !real(a[2], &scale)) Py_RETURN_NONE;
        const ScalarType type = a[3] == Py_None ? w->scalar_type() : a[3] == Py_True ? F32 : BF16;
        at::DimVector shape(ids->sizes());
        shape.push_back(w->size(1));
        at::Tensor out = make(shape, type, *w);
        const int rc = unlocked([&] {
            return lib.moe_embed(pi, ids->scalar_type() != I32, pw, w->scalar_type() == F32, ids->numel(), w->size(0),
                                 w->size(1), scale, ptr(out), type == F32, static_cast<int32_t*>(st), stream());
        });
        return rc ? code(rc) : wrap(out);
    });
}

// embed_backward(ids, dy, V, scale, out or None, fp32, accumulate, status)
PyObject* embed_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args c;
        const at::Tensor* dy = n == 8 && lib.moe_embed_backward ? tensor(a[1]) : nullptr;
        const void* pi = nullptr;
        const at::Tensor* ids = dy ? ids_of(c, a[0], &pi) : nullptr;
        if (!ids || !one_of(dy->scalar_type()) || dy->dim() != ids->dim() + 1) Py_RETURN_NONE;
        const int64_t d = dy->size(-1);
        if (!fits(d) || dy->sizes().slice(0, ids->dim()) != ids->sizes()) Py_RETURN_NONE;
        int V;
        float scale;
        if (!integer(a[2], &V) || V < 1 || !real(a[3], &scale)) Py_RETURN_NONE;
        bool f32, acc;
        if (!truth(a[5], &f32) || !truth(a[6], &acc)) Py_RETURN_NONE;
        const void* py = c.plain(*dy, dy->scalar_type());
        c.opt(a[4], f32 ? F32 : BF16, {V, d});
        void* st = c.opt(a[7], I32, {1});
        if (!c.ok || (acc && a[4] == Py_None)) Py_RETURN_NONE;
        const size_t need = lib.moe_embed_backward_workspace_size(ids->numel(), V, d);
        at::Tensor ws, out = a[4] == Py_None ? make({V, d}, f32 ? F32 : BF16, *dy) : *tensor(a[4]);
        if (need) ws = make({static_cast<int64_t>(need)}, ScalarType::Byte, *dy);
        const int rc = unlocked([&] {
            return lib.moe_embed_backward(pi, ids->scalar_type() != I32, py, dy->scalar_type() == F32, ids->numel(), V, d,
                                          scale, ptr(out), f32, acc, ptr(ws), need, static_cast<int32_t*>(st), stream());
        });
        if (rc) return code(rc);
        if (a[4] == Py_None) return wrap(out);
        touch(out);
        Py_INCREF(a[4]);
        return a[4];
    });
}

// wrote(tensors, lists of tensors or None ...)
PyObject* wrote(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        for (Py_ssize_t k = 0; k < n; ++k) {
            const bool many = PyList_Check(a[k]) || PyTuple_Check(a[k]);
            const Py_ssize_t count = many ? PySequence_Fast_GET_SIZE(a[k]) : 1;
            for (Py_ssize_t i = 0; i < count; ++i) {
                const at::Tensor* t = tensor(many ? PySequence_Fast_GET_ITEM(a[k], i) : a[k]);
                if (t) touch(*t);
            }
        }
        Py_RETURN_NONE;
    });
}

// init(path of libmoe.so)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    const char* path = n == 1 ? PyUnicode_AsUTF8(a[0]) : nullptr;
    if (!path) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "init(path)");
        return nullptr;
    }
    void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!h) {
        PyErr_SetString(PyExc_OSError, dlerror());
        return nullptr;
    }
#define X(name)                                                        \
    lib.name = reinterpret_cast<decltype(&::name)>(dlsym(h, #name));   \
    if (!lib.name) {                                                   \
        PyErr_SetString(PyExc_OSError, #name " is missing");           \
        return nullptr;                                                \
    }
    MOE_FAST_CALLS(X)
#undef X
#define X(name) lib.name = reinterpret_cast<decltype(&::name)>(dlsym(h, #name));
    MOE_FAST_MORE_CALLS(X)
#undef X
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init),          FAST(swiglu),     FAST(swiglu_backward),  FAST(block_norm),
                         FAST(block_norm_backward), FAST(grouped_mm), FAST(grouped_mm_wgrad), FAST(adamw_step),
                         FAST(wrote),
                         FAST(route_scores),  FAST(route_scores_backward), FAST(layer_norm), FAST(layer_norm_backward),
                         FAST(dropout),       FAST(embed),      FAST(embed_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the torch whose headers this was compiled against (MOE_TORCH_VERSION, from the build).
PyMODINIT_FUNC PyInit__moe_fast() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", MOE_TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
