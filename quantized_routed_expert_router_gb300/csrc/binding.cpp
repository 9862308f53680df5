// binding.cpp - the Python side of the calls around the experts: takes torch
// tensors apart, checks shapes, types, layouts and devices, and makes the C
// call on the tensors' device and its current stream.
//
// The same checks written in Python took 4 of the 7 microseconds of a small
// call (0.4 a tensor); here they take about 0.1 in all.  Functions take
// positional arguments (the documented signatures stand in __init__.py) and
// return the moe_status; a tensor that does not fit raises ValueError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <initializer_list>
#include <string>

#include "moe.h"

namespace {

using at::ScalarType;

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(const std::string &text) {
    PyErr_SetString(PyExc_ValueError, text.c_str());
    throw Refused();
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// a tensor argument; null for None where that is allowed
const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": want a tensor" + (optional ? " or None" : ""));
    return &THPVariable_Unpack(o);
}

std::string types_text(std::initializer_list<ScalarType> types) {
    std::string t;
    for (const ScalarType s : types) t += (t.empty() ? "" : " or ") + std::string(at::toString(s));
    return t;
}

// the tensor that the others are held against: contiguous, `dims` dimensions
void lead(const at::Tensor &t, const char *name, int dims, std::initializer_list<ScalarType> types, const char *shape) {
    bool ok = t.dim() == dims && t.is_contiguous(), typed = false;
    for (const ScalarType s : types) typed = typed || t.scalar_type() == s;
    if (!ok || !typed) refuse(std::string(name) + ": want a contiguous " + types_text(types) + " tensor " + shape);
}

// address of a contiguous tensor of this shape and one of these types on the lead's device; null for None
void *expect(PyObject *o, const char *name, at::IntArrayRef shape, std::initializer_list<ScalarType> types, int dev,
             const at::Tensor **out = nullptr) {
    const at::Tensor *t = tensor(o, name, true);
    if (out) *out = t;
    if (!t) return nullptr;
    bool typed = false;
    for (const ScalarType s : types) typed = typed || t->scalar_type() == s;
    if (!typed || t->sizes() != shape || !t->is_contiguous() || t->get_device() != dev)
        refuse(std::string(name) + ": want a contiguous " + types_text(types) + " tensor " + shape_text(shape) +
               " on device " + std::to_string(dev) + ", got " + at::toString(t->scalar_type()) + " " +
               shape_text(t->sizes()) + (t->is_contiguous() ? "" : ", not contiguous,") + " on device " +
               std::to_string(t->get_device()));
    return t->data_ptr();
}

struct Bytes {
    void *p;
    size_t n;
};
// a workspace or record buffer: any type, contiguous, on the lead's device
Bytes buffer(PyObject *o, const char *name, int dev) {
    const at::Tensor *t = tensor(o, name, true);
    if (!t) return {nullptr, 0};
    if (t->get_device() != dev || !t->is_contiguous())
        refuse(std::string(name) + ": want a contiguous tensor on device " + std::to_string(dev));
    return {t->data_ptr(), (size_t)t->nbytes()};
}

int size_of(int64_t n) { return n > INT_MAX ? -1 : (int)n; }   // -1: the C call refuses it

int integer(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < INT_MIN || v > INT_MAX) refuse(std::string(name) + ": out of range");
    return (int)v;
}

float real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}

moe_dtype dtype_of(const at::Tensor *t) {
    return t && t->scalar_type() == ScalarType::BFloat16 ? MOE_DT_BF16 : MOE_DT_F32;
}

// makes call(stream) with `dev` current, on `stream` (a torch stream or None: the current one), without the GIL
template <typename F>
PyObject *launch(const char *name, int dev, PyObject *stream, F call) {
    if (dev < 0) refuse(std::string(name) + ": tensors must be on a CUDA device");
    cudaStream_t s;
    if (stream == Py_None) {
        s = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else {
        PyObject *index = PyObject_GetAttrString(stream, "device_index");
        const long on = index ? PyLong_AsLong(index) : -1;
        Py_XDECREF(index);
        PyObject *handle = PyErr_Occurred() ? nullptr : PyObject_GetAttrString(stream, "cuda_stream");
        s = handle ? (cudaStream_t)PyLong_AsVoidPtr(handle) : nullptr;
        Py_XDECREF(handle);
        if (PyErr_Occurred()) throw Refused();
        if (on != dev) refuse(std::string(name) + ": the stream belongs to another device than the tensors");
    }
    moe_status status;
    {
        const c10::cuda::OptionalCUDAGuard guard((c10::DeviceIndex)dev);
        Py_BEGIN_ALLOW_THREADS;
        status = call(s);
        Py_END_ALLOW_THREADS;
    }
    return PyLong_FromLong((long)status);
}

// runs `body`, turning what it throws into Python exceptions
template <typename F>
PyObject *entry(Py_ssize_t have, Py_ssize_t want, F body) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "want %zd arguments, got %zd", want, have);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

constexpr auto F32 = ScalarType::Float;
constexpr auto BF16 = ScalarType::BFloat16;
constexpr auto I32 = ScalarType::Int;
constexpr auto E4M3 = ScalarType::Float8_e4m3fn;
constexpr auto U8 = ScalarType::Byte;

int64_t groups(int64_t n) { return (n + MOE_FP8_GROUP - 1) / MOE_FP8_GROUP; }

// x, residual, weight, eps, residual_out, y, xq, x8, x8_scale, stream
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 10, [&] {
        const at::Tensor &x = *tensor(a[0], "x");
        lead(x, "x", 2, {F32, BF16}, "[T, n]");
        const int64_t T = x.size(0), n = x.size(1);
        const int dev = (int)x.get_device();
        const auto shape = x.sizes();
        const ScalarType same = x.scalar_type();
        void *r = expect(a[1], "residual", shape, {same}, dev);
        void *w = expect(a[2], "weight", {n}, {F32}, dev);
        const float eps = real(a[3]);
        void *ro = expect(a[4], "residual_out", shape, {same}, dev);
        const at::Tensor *yt;
        void *y = expect(a[5], "y", shape, {F32, BF16}, dev, &yt);
        const Bytes xq = buffer(a[6], "xq", dev);
        const int Ti = size_of(T), ni = size_of(n);
        const size_t need = ni > 0 ? (size_t)T * moe_q8_row_bytes(ni) : 0;
        if (a[6] != Py_None && xq.n < need) refuse("xq: want at least " + std::to_string(need) + " bytes");
        void *x8 = expect(a[7], "x8", shape, {E4M3, U8}, dev);
        void *sc = expect(a[8], "x8_scale", {T, groups(n)}, {F32}, dev);
        return launch("moe_add_rmsnorm", dev, a[9], [&](cudaStream_t s) {
            return moe_add_rmsnorm(x.data_ptr(), r, (const float *)w, eps, Ti, ni, dtype_of(&x), ro, y, dtype_of(yt), xq.p,
                                   x8, (float *)sc, s);
        });
    });
}

// ids, E, ws, counts, offsets, rows, pos, stream
PyObject *expert_order(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 8, [&] {
        const at::Tensor &ids = *tensor(a[0], "ids");
        lead(ids, "ids", 2, {I32}, "[T, k]");
        const int64_t T = ids.size(0), k = ids.size(1);
        const int dev = (int)ids.get_device(), E = integer(a[1], "E");
        const Bytes ws = buffer(a[2], "ws", dev);
        void *counts = expect(a[3], "counts", {E}, {I32}, dev);
        void *offsets = expect(a[4], "offsets", {(int64_t)E + 1}, {I32}, dev);
        void *rows = expect(a[5], "rows", {T * k}, {I32}, dev);
        void *pos = expect(a[6], "pos", ids.sizes(), {I32}, dev);
        return launch("moe_expert_order", dev, a[7], [&](cudaStream_t s) {
            return moe_expert_order((const int32_t *)ids.data_ptr(), size_of(T), size_of(k), E, (int32_t *)counts,
                                    (int32_t *)offsets, (int32_t *)rows, (int32_t *)pos, ws.p, ws.n, s);
        });
    });
}

// logits, counts, k, gating, alpha, ws, loss, dlogits, valid, grad_loss, stream
PyObject *balance_loss(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 11, [&] {
        const at::Tensor &l = *tensor(a[0], "logits");
        lead(l, "logits", 2, {F32, BF16}, "[T, E]");
        const int64_t T = l.size(0), E = l.size(1);
        const int dev = (int)l.get_device();
        void *counts = expect(a[1], "counts", {E}, {I32}, dev);
        const int k = integer(a[2], "k"), gating = integer(a[3], "gating");
        const float alpha = real(a[4]);
        const Bytes ws = buffer(a[5], "ws", dev);
        void *loss = expect(a[6], "loss", {1}, {F32}, dev);
        void *d = expect(a[7], "dlogits", l.sizes(), {l.scalar_type()}, dev);
        void *valid = expect(a[8], "valid", {T}, {U8, ScalarType::Bool}, dev);
        void *scale = expect(a[9], "grad_loss", {1}, {F32}, dev);
        return launch("moe_balance_loss", dev, a[10], [&](cudaStream_t s) {
            return moe_balance_loss(l.data_ptr(), dtype_of(&l), (const int32_t *)counts, (const uint8_t *)valid, size_of(T),
                                    size_of(E), k, (moe_gating)gating, alpha, (const float *)scale, (float *)loss, d, ws.p,
                                    ws.n, s);
        });
    });
}

// x8, x_scale, w, w_scale, y, ws, offsets, rows, stream
PyObject *fp8_matmul(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 9, [&] {
        const at::Tensor &x = *tensor(a[0], "x8"), &w = *tensor(a[2], "w"), &y = *tensor(a[4], "y");
        lead(x, "x8", 2, {E4M3, U8}, "[X, K]");
        if ((w.dim() != 2 && w.dim() != 3) || y.dim() != 2) refuse("w: want [N, K] or [G, N, K]; y: [M, N]");
        const int64_t X = x.size(0), K = x.size(1), N = w.size(-2), M = y.size(0), G = w.dim() == 3 ? w.size(0) : 1;
        const int dev = (int)x.get_device();
        const int64_t ws3[3] = {G, N, K}, sc3[3] = {G, groups(N), groups(K)};
        const size_t skip = w.dim() == 3 ? 0 : 1;
        void *xs = expect(a[1], "x_scale", {X, groups(K)}, {F32}, dev);
        void *wp = expect(a[2], "w", at::IntArrayRef(ws3 + skip, 3 - skip), {E4M3, U8}, dev);
        void *sc = expect(a[3], "w_scale", at::IntArrayRef(sc3 + skip, 3 - skip), {F32}, dev);
        void *yp = expect(a[4], "y", {M, N}, {F32, BF16}, dev);
        const Bytes ws = buffer(a[5], "ws", dev);
        void *offsets = expect(a[6], "offsets", {G + 1}, {I32}, dev);
        void *rows = expect(a[7], "rows", {M}, {I32}, dev);
        return launch("moe_fp8_matmul", dev, a[8], [&](cudaStream_t s) {
            return moe_fp8_matmul(x.data_ptr(), (const float *)xs, size_of(X), (const int32_t *)rows, size_of(M),
                                  (const int32_t *)offsets, size_of(G), wp, (const float *)sc, size_of(N), size_of(K), yp,
                                  dtype_of(&y), ws.p, ws.n, s);
        });
    });
}

// logits, gating, renormalize, ids, weights, valid, stream
PyObject *topk(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 7, [&] {
        const at::Tensor &l = *tensor(a[0], "logits"), &ids = *tensor(a[3], "ids");
        lead(l, "logits", 2, {F32, BF16}, "[T, E]");
        lead(ids, "ids", 2, {I32}, "[T, k]");
        const int64_t T = l.size(0), E = l.size(1), k = ids.size(1);
        const int dev = (int)l.get_device(), gating = integer(a[1], "gating"), renorm = integer(a[2], "renormalize");
        void *out = expect(a[3], "ids", {T, k}, {I32}, dev);
        void *w = expect(a[4], "weights", {T, k}, {F32}, dev);
        void *valid = expect(a[5], "valid", {T}, {U8, ScalarType::Bool}, dev);
        return launch("moe_topk", dev, a[6], [&](cudaStream_t s) {
            return moe_topk(l.data_ptr(), dtype_of(&l), (const uint8_t *)valid, size_of(T), size_of(E), size_of(k),
                            (moe_gating)gating, renorm, (int32_t *)out, (float *)w, s);
        });
    });
}

// logits, ids, dweights, gating, renormalize, dlogits, addend, stream
PyObject *topk_grad(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 8, [&] {
        const at::Tensor &l = *tensor(a[0], "logits"), &ids = *tensor(a[1], "ids");
        lead(l, "logits", 2, {F32, BF16}, "[T, E]");
        lead(ids, "ids", 2, {I32}, "[T, k]");
        const int64_t T = l.size(0), E = l.size(1), k = ids.size(1);
        const int dev = (int)l.get_device();
        void *in = expect(a[1], "ids", {T, k}, {I32}, dev);
        void *dw = expect(a[2], "dweights", {T, k}, {F32}, dev);
        const int gating = integer(a[3], "gating"), renorm = integer(a[4], "renormalize");
        void *d = expect(a[5], "dlogits", l.sizes(), {l.scalar_type()}, dev);
        void *add = expect(a[6], "addend", l.sizes(), {l.scalar_type()}, dev);
        return launch("moe_topk_grad", dev, a[7], [&](cudaStream_t s) {
            return moe_topk_grad(l.data_ptr(), dtype_of(&l), (const int32_t *)in, (const float *)dw, size_of(T), size_of(E),
                                 size_of(k), (moe_gating)gating, renorm, add, d, s);
        });
    });
}

// x, pos, xs, stream
PyObject *dispatch_rows(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 4, [&] {
        const at::Tensor &x = *tensor(a[0], "x"), &pos = *tensor(a[1], "pos"), &xs = *tensor(a[2], "xs");
        lead(x, "x", 2, {F32, BF16}, "[T, n]");
        lead(pos, "pos", 2, {I32}, "[T, k]");
        lead(xs, "xs", 2, {x.scalar_type()}, "[M, n]");
        const int64_t T = x.size(0), n = x.size(1), k = pos.size(1), M = xs.size(0);
        const int dev = (int)x.get_device();
        void *p = expect(a[1], "pos", {T, k}, {I32}, dev);
        void *to = expect(a[2], "xs", {M, n}, {x.scalar_type()}, dev);
        return launch("moe_dispatch_rows", dev, a[3], [&](cudaStream_t s) {
            return moe_dispatch_rows(x.data_ptr(), dtype_of(&x), (const int32_t *)p, size_of(T), size_of(k), size_of(n),
                                     size_of(M), to, s);
        });
    });
}

// o, pos, y, weights, addend, stream
PyObject *combine_rows(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 6, [&] {
        const at::Tensor &o = *tensor(a[0], "o"), &pos = *tensor(a[1], "pos"), &y = *tensor(a[2], "y");
        lead(o, "o", 2, {F32, BF16}, "[M, n]");
        lead(pos, "pos", 2, {I32}, "[T, k]");
        lead(y, "y", 2, {F32, BF16}, "[T, n]");
        const int64_t T = pos.size(0), k = pos.size(1), n = o.size(1), M = o.size(0);
        const int dev = (int)o.get_device();
        void *p = expect(a[1], "pos", {T, k}, {I32}, dev);
        void *out = expect(a[2], "y", {T, n}, {F32, BF16}, dev);
        void *w = expect(a[3], "weights", {T, k}, {F32}, dev);
        void *add = expect(a[4], "addend", {T, n}, {y.scalar_type()}, dev);
        return launch("moe_combine_rows", dev, a[5], [&](cudaStream_t s) {
            return moe_combine_rows(o.data_ptr(), dtype_of(&o), (const int32_t *)p, (const float *)w, size_of(T), size_of(k),
                                    size_of(n), size_of(M), add, out, dtype_of(&y), s);
        });
    });
}

// dy, pos, weights, o, d_o, dweights, stream
PyObject *combine_grad(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 7, [&] {
        const at::Tensor &dy = *tensor(a[0], "dy"), &pos = *tensor(a[1], "pos");
        lead(dy, "dy", 2, {F32, BF16}, "[T, n]");
        lead(pos, "pos", 2, {I32}, "[T, k]");
        const int64_t T = dy.size(0), n = dy.size(1), k = pos.size(1);
        const int dev = (int)dy.get_device();
        const at::Tensor *o = tensor(a[3], "o", true), *d = tensor(a[4], "do", true);
        const at::Tensor *rows = o ? o : d;   // whose rows the places are
        if (!rows) refuse("do: want do, or dweights with o");
        lead(*rows, o ? "o" : "do", 2, {F32, BF16}, "[M, n]");
        const int64_t M = rows->size(0);
        void *p = expect(a[1], "pos", {T, k}, {I32}, dev);
        void *w = expect(a[2], "weights", {T, k}, {F32}, dev);
        void *op = expect(a[3], "o", {M, n}, {rows->scalar_type()}, dev);
        void *dp = expect(a[4], "do", {M, n}, {rows->scalar_type()}, dev);
        void *dw = expect(a[5], "dweights", {T, k}, {F32}, dev);
        return launch("moe_combine_grad", dev, a[6], [&](cudaStream_t s) {
            return moe_combine_grad(dy.data_ptr(), dtype_of(&dy), (const int32_t *)p, (const float *)w, size_of(T),
                                    size_of(k), size_of(n), size_of(M), op, dtype_of(rows), dp, (float *)dw, s);
        });
    });
}

// x, w, y, ws, act, bias, residual, z, offsets, rows, transposed, stream
PyObject *matmul(PyObject *, PyObject *const *a, Py_ssize_t have) {
    return entry(have, 12, [&] {
        const at::Tensor &x = *tensor(a[0], "x"), &w = *tensor(a[1], "w"), &y = *tensor(a[2], "y");
        lead(x, "x", 2, {BF16}, "[X, K]");
        lead(y, "y", 2, {F32, BF16}, "[M, N] ([M, 2 N] with ACT_SWIGLU_GRAD)");
        if (w.dim() != 2 && w.dim() != 3) refuse("w: want [N, K] or [G, N, K] (transposed: [K, N] or [G, K, N])");
        const int act = integer(a[4], "act"), transposed = integer(a[10], "transposed");
        const int64_t X = x.size(0), K = x.size(1), M = y.size(0), G = w.dim() == 3 ? w.size(0) : 1;
        const int64_t wide = w.size(transposed ? -1 : -2);   // columns of the product
        if (act == MOE_ACT_SWIGLU && wide % 2) refuse("w: want gate rows and as many up rows");
        const int64_t N = act == MOE_ACT_SWIGLU ? wide / 2 : wide, yn = act == MOE_ACT_SWIGLU_GRAD ? 2 * N : N;
        const int64_t zn = act == MOE_ACT_SWIGLU || act == MOE_ACT_SWIGLU_GRAD ? 2 * N : N;
        const int dev = (int)x.get_device();
        const int64_t ws3[3] = {G, transposed ? K : wide, transposed ? wide : K}, b2[2] = {G, wide};
        const size_t skip = w.dim() == 3 ? 0 : 1;
        void *wp = expect(a[1], "w", at::IntArrayRef(ws3 + skip, 3 - skip), {BF16}, dev);
        void *yp = expect(a[2], "y", {M, yn}, {F32, BF16}, dev);
        const Bytes ws = buffer(a[3], "ws", dev);
        void *bias = expect(a[5], "bias", at::IntArrayRef(b2 + skip, 2 - skip), {F32}, dev);
        void *res = expect(a[6], "residual", {M, N}, {y.scalar_type()}, dev);
        void *z = expect(a[7], "z", {M, zn}, {y.scalar_type()}, dev);
        void *offsets = expect(a[8], "offsets", {G + 1}, {I32}, dev);
        void *rows = expect(a[9], "rows", {M}, {I32}, dev);
        return launch("moe_matmul", dev, a[11], [&](cudaStream_t s) {
            return moe_matmul(x.data_ptr(), size_of(X), (const int32_t *)rows, size_of(M), (const int32_t *)offsets,
                              size_of(G), wp, transposed, (const float *)bias, (moe_act)act, res, z, size_of(N), size_of(K),
                              yp, dtype_of(&y), ws.p, ws.n, s);
        });
    });
}

#define CALL(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(add_rmsnorm), CALL(expert_order), CALL(balance_loss), CALL(fp8_matmul), CALL(topk),
                         CALL(topk_grad), CALL(dispatch_rows), CALL(combine_rows), CALL(combine_grad), CALL(matmul), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
    PyObject *m = PyModule_Create(&module);
    // what this object was compiled against, as the build names it
    if (m && PyModule_AddStringConstant(m, "built_for", CALLS_STAMP) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
