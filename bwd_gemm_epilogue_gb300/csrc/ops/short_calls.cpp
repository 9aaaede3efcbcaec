// short_calls.cpp -- a Python module with the usual calls of the operators in swiglu_ops.h,
// swiglu_tokens.h and swiglu_moe.h over torch tensors, for binding.py.
//
// On the device these calls can be shorter than the 20 to 30 us that Python takes to check a call's
// tensors, make its outputs and pass its 20 arguments (a norm of 16 rows: 4 us), so the usual call,
// every tensor as it should be and every output new, is made here.  Anything else returns None, and
// binding.py makes the call, or explains what is wrong with it.  A status other than 0 is returned as
// an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "swiglu_moe.h"
#include "swiglu_ops.h"
#include "swiglu_tokens.h"

namespace {

using at::Tensor;

// The caller's tensor, or nullptr; `none`: whether None is allowed (then also nullptr).
struct Arg {
    const Tensor* t = nullptr;
    bool ok = false;
    Arg(PyObject* o, bool none) {
        if (o == Py_None) {
            ok = none;
        } else if (THPVariable_Check(o)) {
            t = &THPVariable_Unpack(o);
            ok = t->defined() && t->is_cuda() && t->layout() == at::kStrided;
        }
    }
    void* data() const { return t ? t->data_ptr() : nullptr; }
    int64_t stride() const { return t ? t->stride(0) : 0; }
};

int code_of(at::ScalarType type) {
    return type == at::kBFloat16 ? SWIGLU_BF16 : type == at::kHalf ? SWIGLU_FP16 : type == at::kFloat ? SWIGLU_FP32 : -1;
}

// [M, D] rows like x's, each contiguous, none overlapping.
bool rows_like(const Arg& a, const Tensor& x) {
    if (!a.t) return true;
    const Tensor& t = *a.t;
    return t.dim() == 2 && t.size(0) == x.size(0) && t.size(1) == x.size(1) && t.stride(1) == 1 && t.stride(0) >= t.size(1) &&
           t.scalar_type() == x.scalar_type() && t.device() == x.device();
}

bool contiguous(const Arg& a, at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    if (!a.t) return true;
    return a.t->sizes() == shape && a.t->scalar_type() == type && a.t->device() == device && a.t->is_contiguous();
}

Tensor fresh(at::IntArrayRef shape, at::ScalarType type, at::Device device) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
}

bool on_current_device(at::Device d) { return d.index() == c10::cuda::current_device(); }
void* stream_of(at::Device d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// A tuple of tensors, and objects the caller passed.
PyObject* tuple_of(std::initializer_list<PyObject*> items) {
    PyObject* r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
    return r;
}
PyObject* share(PyObject* o) {
    Py_INCREF(o);
    return o;
}

// A launch can wait for room in the stream's queue: other threads run meanwhile.
struct WithoutGil {
    PyThreadState* state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
};
template <class F>
int released(const F& f) {
    const WithoutGil r;
    return f();
}

// A C++ exception (no memory for an output, say) as the Python exception that torch makes of it.
template <class F>
PyObject* guarded(const F& f) {
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// (x, gamma, beta, eps, residual) -> (y, s, mean, rstd)
PyObject* layer_norm_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) Py_RETURN_NONE;
        const Arg x(args[0], false), gamma(args[1], true), beta(args[2], true), r(args[4], true);
        const double eps = PyFloat_Check(args[3]) ? PyFloat_AS_DOUBLE(args[3]) : -1.0;
        if (!x.ok || !gamma.ok || !beta.ok || !r.ok || !(eps >= 0.0)) Py_RETURN_NONE;
        const Tensor& t = *x.t;
        const int code = code_of(t.scalar_type());
        if (code < 0 || !rows_like(x, t) || !rows_like(r, t) || !on_current_device(t.device())) Py_RETURN_NONE;
        const int64_t M = t.size(0), D = t.size(1);
        const at::ScalarType wtype = gamma.t ? gamma.t->scalar_type() : beta.t ? beta.t->scalar_type() : t.scalar_type();
        if ((wtype != t.scalar_type() && wtype != at::kFloat) || !contiguous(gamma, {D}, wtype, t.device()) ||
            !contiguous(beta, {D}, wtype, t.device()))
            Py_RETURN_NONE;
        Tensor y = fresh({M, D}, t.scalar_type(), t.device()), s;
        if (r.t) s = fresh({M, D}, t.scalar_type(), t.device());
        Tensor mean = fresh({M}, at::kFloat, t.device()), rstd = fresh({M}, at::kFloat, t.device());
        const int st = released([&] {
            return swiglu_mlp_layer_norm_fwd(x.data(), x.stride(), r.data(), r.stride(), gamma.data(), beta.data(), y.data_ptr(), D,
                r.t ? s.data_ptr() : nullptr, r.t ? D : 0, mean.data_ptr<float>(),
                rstd.data_ptr<float>(), M, D, (float)eps, code, code_of(wtype), stream_of(t.device()));
        });
        if (st) return PyLong_FromLong(st);
        PyObject* ps = r.t ? THPVariable_Wrap(std::move(s)) : share(args[0]);
        return tuple_of({THPVariable_Wrap(std::move(y)), ps, THPVariable_Wrap(std::move(mean)), THPVariable_Wrap(std::move(rstd))});
    });
}

// (dy, s, gamma, mean, rstd, dskip) -> (dx, dgamma, dbeta)
PyObject* layer_norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 6) Py_RETURN_NONE;
        const Arg dy(args[0], false), s(args[1], false), gamma(args[2], true), mean(args[3], false), rstd(args[4], false), skip(args[5], true);
        if (!dy.ok || !s.ok || !gamma.ok || !mean.ok || !rstd.ok || !skip.ok) Py_RETURN_NONE;
        const Tensor& t = *s.t;
        const int code = code_of(t.scalar_type());
        if (code < 0 || !rows_like(s, t) || !rows_like(dy, t) || !rows_like(skip, t) || !on_current_device(t.device())) Py_RETURN_NONE;
        const int64_t M = t.size(0), D = t.size(1);
        const at::ScalarType wtype = gamma.t ? gamma.t->scalar_type() : t.scalar_type();
        if ((wtype != t.scalar_type() && wtype != at::kFloat) || !contiguous(gamma, {D}, wtype, t.device()) ||
            !contiguous(mean, {M}, at::kFloat, t.device()) || !contiguous(rstd, {M}, at::kFloat, t.device()))
            Py_RETURN_NONE;
        const int64_t need = std::max<int64_t>(16, (int64_t)swiglu_mlp_layer_norm_bwd_workspace_size(M, D));
        Tensor dx = fresh({M, D}, t.scalar_type(), t.device()), dgamma = fresh({D}, wtype, t.device()), dbeta = fresh({D}, wtype, t.device());
        Tensor workspace = fresh({need}, at::kByte, t.device());
        const int st = released([&] {
            return swiglu_mlp_layer_norm_bwd(dy.data(), dy.stride(), s.data(), s.stride(), gamma.data(), mean.t->data_ptr<float>(),
                rstd.t->data_ptr<float>(), skip.data(), skip.stride(), dx.data_ptr(), D, dgamma.data_ptr(),
                dbeta.data_ptr(), M, D, code, code_of(wtype), workspace.data_ptr(), (size_t)need,
                stream_of(t.device()));
        });
        if (st) return PyLong_FromLong(st);
        return tuple_of({THPVariable_Wrap(std::move(dx)), THPVariable_Wrap(std::move(dgamma)), THPVariable_Wrap(std::move(dbeta))});
    });
}

// ([gradients], [outputs] or None: the norm alone, max_norm, eps) -> norm; the same list twice: in place
PyObject* clip_grads(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 4 || !PyList_Check(args[0]) || !(PyList_Check(args[1]) || args[1] == Py_None)) Py_RETURN_NONE;
        const double max_norm = PyFloat_AsDouble(args[2]), eps = PyFloat_AsDouble(args[3]);
        if (PyErr_Occurred()) return nullptr;
        const Py_ssize_t count = PyList_GET_SIZE(args[0]);
        const bool write = args[1] != Py_None;
        if (count == 0 || (write && PyList_GET_SIZE(args[1]) != count) || (write && (!(max_norm >= 0.0) || !(eps >= 0.0)))) Py_RETURN_NONE;
        std::vector<const void*> in(count);
        std::vector<void*> out(write ? count : 0);
        std::vector<int64_t> counts(count);
        std::vector<int> types(count);
        c10::optional<at::Device> device;
        for (Py_ssize_t i = 0; i < count; ++i) {
            const Arg g(PyList_GET_ITEM(args[0], i), false);
            if (!g.ok || !g.t->is_contiguous()) Py_RETURN_NONE;
            if (!device) device = g.t->device();
            types[i] = code_of(g.t->scalar_type());
            if (types[i] < 0 || g.t->device() != *device) Py_RETURN_NONE;
            in[i] = g.data();
            counts[i] = g.t->numel();
            if (!write) continue;
            const Arg o(PyList_GET_ITEM(args[1], i), false);
            if (!o.ok || !o.t->is_contiguous() || o.t->device() != *device || o.t->scalar_type() != g.t->scalar_type() ||
                o.t->numel() != counts[i])
                Py_RETURN_NONE;
            out[i] = o.data();
        }
        if (!on_current_device(*device)) Py_RETURN_NONE;
        const int64_t need = std::max<int64_t>(16, (int64_t)swiglu_mlp_clip_grads_workspace_size(count));
        Tensor norm = fresh({}, at::kFloat, *device), workspace = fresh({need}, at::kByte, *device);
        const int st = released([&] {
            return swiglu_mlp_clip_grads(in.data(), write ? out.data() : nullptr, counts.data(), types.data(), count, (float)max_norm,
                (float)eps, norm.data_ptr<float>(), workspace.data_ptr(), (size_t)need, stream_of(*device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(norm));
    });
}

// (x, Wr, W1, W2, top_k, renormalize, residual) -> (y, ids, gates)
PyObject* moe_routed_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 7 || !PyLong_Check(args[4])) Py_RETURN_NONE;
        const Arg x(args[0], false), wr(args[1], false), w1(args[2], false), w2(args[3], false), r(args[6], true);
        int over = 0;
        const int64_t k = PyLong_AsLongLongAndOverflow(args[4], &over);
        const int renorm = PyObject_IsTrue(args[5]);
        if (renorm < 0) return nullptr;    // a value without a truth: its own error
        if (!x.ok || !wr.ok || !w1.ok || !w2.ok || !r.ok || over || k <= 0 || x.t->dim() != 2 || w2.t->dim() != 3) Py_RETURN_NONE;
        const at::Device device = x.t->device();
        const at::ScalarType bf = at::kBFloat16, rtype = wr.t->scalar_type();
        const int64_t T = x.t->size(0), D = x.t->size(1), E = w2.t->size(0), Dout = w2.t->size(1), H = w2.t->size(2);
        if ((rtype != bf && rtype != at::kFloat) || !contiguous(x, {T, D}, bf, device) || !contiguous(wr, {E, D}, rtype, device) ||
            !contiguous(w1, {E, 2 * H, D}, bf, device) || !contiguous(w2, {E, Dout, H}, bf, device) ||
            !contiguous(r, {T, Dout}, bf, device) || !on_current_device(device))
            Py_RETURN_NONE;
        const int64_t need = std::max<int64_t>(16, (int64_t)swiglu_moe_routed_fwd_workspace_size(T, H, Dout, k));
        if (k > E || k > 1024) Py_RETURN_NONE;
        Tensor y = fresh({T, Dout}, bf, device), ids = fresh({T, k}, at::kInt, device), gates = fresh({T, k}, at::kFloat, device);
        Tensor workspace = fresh({need}, at::kByte, device);
        const int st = released([&] {
            return swiglu_moe_routed_fwd(x.data(), wr.data(), w1.data(), w2.data(), r.data(), y.data_ptr(), ids.data_ptr<int>(),
                gates.data_ptr<float>(), T, E, D, H, Dout, k, renorm, rtype == at::kFloat,
                workspace.data_ptr(), (size_t)need, stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return tuple_of({THPVariable_Wrap(std::move(y)), THPVariable_Wrap(std::move(ids)), THPVariable_Wrap(std::move(gates))});
    });
}

// ---------------------------------------------------------------- tokens to experts and back

// [M, D] rows of `type`, each contiguous, none overlapping.
bool rows_of(const Arg& a, int64_t M, int64_t D, at::ScalarType type, at::Device device) {
    if (!a.t) return true;
    const Tensor& t = *a.t;
    return t.dim() == 2 && t.size(0) == M && t.size(1) == D && t.stride(1) == 1 && t.stride(0) >= D && t.scalar_type() == type &&
           t.device() == device;
}

// Rows of one of the element types on the current device.
bool rows_alone(const Arg& a, int* code) {
    if (!a.ok || !a.t || a.t->dim() != 2) return false;
    *code = code_of(a.t->scalar_type());
    return *code >= 0 && rows_like(a, *a.t) && on_current_device(a.t->device());
}

bool pairs_of(const Arg& a, int64_t T, int64_t k, at::ScalarType type, at::Device device) {
    return a.ok && a.t && contiguous(a, {T, k}, type, device);
}

// A whole number in 0 .. 2^63 - 1 (larger ones, which are rare, are taken by binding.py).
bool whole(PyObject* o, int64_t* v) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    *v = PyLong_AsLongLongAndOverflow(o, &over);
    return !over && *v >= 0;
}

// (p, seed, offset, step) of a dropout.
struct Mask {
    double p = 0;
    int64_t seed = 0, offset = 0;
    Arg step;
    bool ok;
    Mask(PyObject* const* args, at::Device device) : step(args[3], true) {
        ok = PyFloat_CheckExact(args[0]) && whole(args[1], &seed) && whole(args[2], &offset) && step.ok &&
             (!step.t || (step.t->dim() == 0 && step.t->scalar_type() == at::kLong && step.t->device() == device));
        if (ok) p = PyFloat_AS_DOUBLE(args[0]);
    }
    const int64_t* at() const { return static_cast<const int64_t*>(step.data()); }
};

// (logits, top_k, renormalize) -> (ids, gates)
PyObject* moe_gate_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) Py_RETURN_NONE;
        const Arg l(args[0], false);
        int64_t k;
        int code;
        const int renorm = PyObject_IsTrue(args[2]);
        if (renorm < 0) return nullptr;
        if (!whole(args[1], &k) || !rows_alone(l, &code) || k < 1 || k > l.t->size(1)) Py_RETURN_NONE;
        const int64_t T = l.t->size(0), E = l.t->size(1);
        const at::Device device = l.t->device();
        Tensor ids = fresh({T, k}, at::kInt, device), gates = fresh({T, k}, at::kFloat, device);
        const int st = released([&] {
            return swiglu_moe_gate_fwd(l.data(), l.stride(), ids.data_ptr<int>(), gates.data_ptr<float>(), T, E, k, renorm, code,
                stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return tuple_of({THPVariable_Wrap(std::move(ids)), THPVariable_Wrap(std::move(gates))});
    });
}

// (logits, ids, gates, dgates, renormalize) -> dlogits
PyObject* moe_gate_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 5) Py_RETURN_NONE;
        const Arg l(args[0], false), ids(args[1], false), q(args[2], false), dq(args[3], false);
        int code;
        const int renorm = PyObject_IsTrue(args[4]);
        if (renorm < 0) return nullptr;
        if (!rows_alone(l, &code) || !ids.ok || ids.t->dim() != 2) Py_RETURN_NONE;
        const int64_t T = l.t->size(0), E = l.t->size(1), k = ids.t->size(1);
        const at::Device device = l.t->device();
        if (k < 1 || k > E || !pairs_of(ids, T, k, at::kInt, device) || !pairs_of(q, T, k, at::kFloat, device) ||
            !pairs_of(dq, T, k, at::kFloat, device))
            Py_RETURN_NONE;
        Tensor d = fresh({T, E}, l.t->scalar_type(), device);
        const int st = released([&] {
            return swiglu_moe_gate_bwd(l.data(), l.stride(), ids.t->data_ptr<int>(), q.t->data_ptr<float>(), dq.t->data_ptr<float>(),
                d.data_ptr(), E, T, E, k, renorm, code, stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(d));
    });
}

// (ids, E) -> (counts, pos)
PyObject* moe_sort(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 2) Py_RETURN_NONE;
        const Arg ids(args[0], false);
        int64_t E;
        if (!whole(args[1], &E) || E > 1024 || !ids.ok || ids.t->scalar_type() != at::kInt || !ids.t->is_contiguous() ||
            !on_current_device(ids.t->device()))
            Py_RETURN_NONE;
        const at::Device device = ids.t->device();
        Tensor counts = fresh({E}, at::kInt, device), pos = fresh(ids.t->sizes(), at::kInt, device);
        const int st = released([&] {
            return swiglu_moe_sort(ids.t->data_ptr<int>(), counts.data_ptr<int>(), pos.data_ptr<int>(), ids.t->numel(), E, stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return tuple_of({THPVariable_Wrap(std::move(counts)), THPVariable_Wrap(std::move(pos))});
    });
}

// (x, pos, n_rows or None: one for each pair) -> rows
PyObject* moe_dispatch_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) Py_RETURN_NONE;
        const Arg x(args[0], false), pos(args[1], false);
        int code;
        if (!rows_alone(x, &code) || !pos.ok || pos.t->dim() != 2) Py_RETURN_NONE;
        const int64_t T = x.t->size(0), D = x.t->size(1), k = pos.t->size(1);
        const at::Device device = x.t->device();
        int64_t rows = T * k;
        if (!pairs_of(pos, T, k, at::kInt, device) || (args[2] != Py_None && !whole(args[2], &rows))) Py_RETURN_NONE;
        Tensor out = fresh({rows, D}, x.t->scalar_type(), device);
        const int st = released([&] {
            return swiglu_moe_dispatch_fwd(x.data(), x.stride(), pos.t->data_ptr<int>(), out.data_ptr(), D, T, D, k, rows, code,
                stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(out));
    });
}

// (drows, pos, add) -> dx
PyObject* moe_dispatch_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 3) Py_RETURN_NONE;
        const Arg d(args[0], false), pos(args[1], false), add(args[2], true);
        int code;
        if (!rows_alone(d, &code) || !pos.ok || pos.t->dim() != 2 || !add.ok) Py_RETURN_NONE;
        const int64_t rows = d.t->size(0), D = d.t->size(1), T = pos.t->size(0), k = pos.t->size(1);
        const at::Device device = d.t->device();
        const at::ScalarType type = d.t->scalar_type(), atype = add.t && add.t->scalar_type() == at::kFloat ? at::kFloat : type;
        if (!pairs_of(pos, T, k, at::kInt, device) || !rows_of(add, T, D, atype, device)) Py_RETURN_NONE;
        Tensor dx = fresh({T, D}, type, device);
        const int st = released([&] {
            return swiglu_moe_dispatch_bwd(d.data(), d.stride(), pos.t->data_ptr<int>(), add.data(), add.stride(), dx.data_ptr(), D, T, D,
                k, rows, code, code_of(atype), stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(dx));
    });
}

// (rows, pos, gates, residual, p, seed, offset, step) -> y
PyObject* moe_combine_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) Py_RETURN_NONE;
        const Arg rows(args[0], false), pos(args[1], false), gates(args[2], false), r(args[3], true);
        int code;
        if (!rows_alone(rows, &code) || !pos.ok || pos.t->dim() != 2 || !r.ok) Py_RETURN_NONE;
        const int64_t R = rows.t->size(0), D = rows.t->size(1), T = pos.t->size(0), k = pos.t->size(1);
        const at::Device device = rows.t->device();
        const at::ScalarType type = rows.t->scalar_type();
        const Mask m(args + 4, device);
        if (!m.ok || !pairs_of(pos, T, k, at::kInt, device) || !pairs_of(gates, T, k, at::kFloat, device) ||
            !rows_of(r, T, D, type, device))
            Py_RETURN_NONE;
        Tensor y = fresh({T, D}, type, device);
        const int st = released([&] {
            return swiglu_moe_combine_fwd(rows.data(), rows.stride(), pos.t->data_ptr<int>(), gates.t->data_ptr<float>(), r.data(),
                r.stride(), y.data_ptr(), D, T, D, k, R, code, m.p, m.seed, m.offset, m.at(), stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(y));
    });
}

// (dy, rows, pos, gates, p, seed, offset, step) -> (drows, dgates)
PyObject* moe_combine_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) Py_RETURN_NONE;
        const Arg dy(args[0], false), rows(args[1], false), pos(args[2], false), gates(args[3], false);
        int code;
        if (!rows_alone(rows, &code) || !pos.ok || pos.t->dim() != 2 || !dy.ok) Py_RETURN_NONE;
        const int64_t R = rows.t->size(0), D = rows.t->size(1), T = pos.t->size(0), k = pos.t->size(1);
        const at::Device device = rows.t->device();
        const at::ScalarType type = rows.t->scalar_type();
        const Mask m(args + 4, device);
        if (!m.ok || !pairs_of(pos, T, k, at::kInt, device) || !pairs_of(gates, T, k, at::kFloat, device) ||
            !rows_of(dy, T, D, type, device))
            Py_RETURN_NONE;
        Tensor drows = fresh({R, D}, type, device), dgates = fresh({T, k}, at::kFloat, device);
        const int st = released([&] {
            return swiglu_moe_combine_bwd(dy.data(), dy.stride(), rows.data(), rows.stride(), pos.t->data_ptr<int>(),
                gates.t->data_ptr<float>(), drows.data_ptr(), D, dgates.data_ptr<float>(), T, D, k, R, code, m.p, m.seed, m.offset,
                m.at(), stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return tuple_of({THPVariable_Wrap(std::move(drows)), THPVariable_Wrap(std::move(dgates))});
    });
}

// (x, residual, p, seed, offset, step) -> y
PyObject* dropout(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 6) Py_RETURN_NONE;
        const Arg x(args[0], false), r(args[1], true);
        int code;
        if (!rows_alone(x, &code) || !r.ok || !rows_like(r, *x.t)) Py_RETURN_NONE;
        const int64_t M = x.t->size(0), D = x.t->size(1);
        const at::Device device = x.t->device();
        const Mask m(args + 2, device);
        if (!m.ok) Py_RETURN_NONE;
        Tensor y = fresh({M, D}, x.t->scalar_type(), device);
        const int st = released([&] {
            return swiglu_mlp_dropout(x.data(), x.stride(), r.data(), r.stride(), y.data_ptr(), D, M, D, code, m.p, m.seed, m.offset,
                m.at(), stream_of(device));
        });
        if (st) return PyLong_FromLong(st);
        return THPVariable_Wrap(std::move(y));
    });
}

PyMethodDef methods[] = {{"layer_norm_fwd", (PyCFunction)(void (*)())layer_norm_fwd, METH_FASTCALL, nullptr},
                         {"layer_norm_bwd", (PyCFunction)(void (*)())layer_norm_bwd, METH_FASTCALL, nullptr},
                         {"clip_grads", (PyCFunction)(void (*)())clip_grads, METH_FASTCALL, nullptr},
                         {"moe_routed_fwd", (PyCFunction)(void (*)())moe_routed_fwd, METH_FASTCALL, nullptr},
                         {"moe_gate_fwd", (PyCFunction)(void (*)())moe_gate_fwd, METH_FASTCALL, nullptr},
                         {"moe_gate_bwd", (PyCFunction)(void (*)())moe_gate_bwd, METH_FASTCALL, nullptr},
                         {"moe_sort", (PyCFunction)(void (*)())moe_sort, METH_FASTCALL, nullptr},
                         {"moe_dispatch_fwd", (PyCFunction)(void (*)())moe_dispatch_fwd, METH_FASTCALL, nullptr},
                         {"moe_dispatch_bwd", (PyCFunction)(void (*)())moe_dispatch_bwd, METH_FASTCALL, nullptr},
                         {"moe_combine_fwd", (PyCFunction)(void (*)())moe_combine_fwd, METH_FASTCALL, nullptr},
                         {"moe_combine_bwd", (PyCFunction)(void (*)())moe_combine_bwd, METH_FASTCALL, nullptr},
                         {"dropout", (PyCFunction)(void (*)())dropout, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_short_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers this was compiled with, which has to be the one that runs.
PyMODINIT_FUNC PyInit__short_calls() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", SWIGLU_TORCH) < 0) Py_CLEAR(m);
    return m;
}
