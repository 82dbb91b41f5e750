// Python extension of the binding: checks lists of torch tensors against the type,
// shape and device that a call will touch, and returns their addresses as one table
// of 64-bit pointers; allocates lists of buffers; and makes the calls that take the
// GPU least (a linear layer, a gated block, clipping, a loss, an AdamW step) whole. The same checks as the
// binding's Python code, at about 20 ns a tensor instead of 500: a call on 8 ranks
// passes 20 to 60 tensors, and a decoded token's product takes the GPU about as long
// as that loop.
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

#include "rtp.h"

namespace {

bool scalar_type(long code, at::ScalarType* out)
{
    if (code != 0 && code != 1) return false;
    *out = code == 0 ? at::kFloat : at::kBFloat16;
    return true;
}

// Empty tensors are never touched: only their type and shape must fit.
bool placed(const at::Tensor& t, long device)
{
    return t.numel() == 0 || (t.get_device() == device && t.is_contiguous());
}

PyObject* pointers(const std::vector<uint64_t>& p)
{
    return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(p.data()), (Py_ssize_t)(p.size() * 8));
}

// table(tensors, shape, dtype code, device) -> bytes, or the index of the first
// tensor that does not fit.
PyObject* table(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 4 || !PyList_Check(args[0]) || !PyTuple_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "table(list, shape, dtype code, device)");
        return nullptr;
    }
    const long code = PyLong_AsLong(args[2]), device = PyLong_AsLong(args[3]);
    at::ScalarType want;
    if (PyErr_Occurred() || !scalar_type(code, &want)) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "table: unknown dtype code");
        return nullptr;
    }
    const Py_ssize_t nd = PyTuple_GET_SIZE(args[1]), n = PyList_GET_SIZE(args[0]);
    int64_t shape[8];
    if (nd > 8) {
        PyErr_SetString(PyExc_ValueError, "table: more than 8 dimensions");
        return nullptr;
    }
    for (Py_ssize_t d = 0; d < nd; ++d) shape[d] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], d));
    if (PyErr_Occurred()) return nullptr;
    const at::IntArrayRef sizes(shape, (size_t)nd);
    std::vector<uint64_t> out((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* o = PyList_GET_ITEM(args[0], i);
        if (!THPVariable_Check(o)) return PyLong_FromSsize_t(i);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() != want || t.sizes() != sizes || !placed(t, device)) return PyLong_FromSsize_t(i);
        out[(size_t)i] = (uint64_t)(uintptr_t)t.data_ptr();
    }
    return pointers(out);
}

// like(tensors, references, device) -> bytes, or the index of the first tensor
// that differs from its reference in type or shape, or is not placed as needed.
PyObject* like(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 3 || !PyList_Check(args[0]) || !PyList_Check(args[1]) ||
        PyList_GET_SIZE(args[0]) != PyList_GET_SIZE(args[1])) {
        PyErr_SetString(PyExc_TypeError, "like(list, list of the same length, device)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[2]);
    if (PyErr_Occurred()) return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(args[0]);
    std::vector<uint64_t> out((size_t)n);
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *a = PyList_GET_ITEM(args[0], i), *b = PyList_GET_ITEM(args[1], i);
        if (!THPVariable_Check(a) || !THPVariable_Check(b)) return PyLong_FromSsize_t(i);
        const at::Tensor &t = THPVariable_Unpack(a), &r = THPVariable_Unpack(b);
        if (t.scalar_type() != r.scalar_type() || t.sizes() != r.sizes() || !placed(t, device)) return PyLong_FromSsize_t(i);
        out[(size_t)i] = (uint64_t)(uintptr_t)t.data_ptr();
    }
    return pointers(out);
}

// buffers(n, shape, dtype code, device) -> list of n new tensors (torch.empty of
// each, on the current stream, without the cost of its Python argument parsing)
PyObject* buffers(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 4 || !PyTuple_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "buffers(n, shape, dtype code, device)");
        return nullptr;
    }
    const Py_ssize_t n = PyLong_AsSsize_t(args[0]), nd = PyTuple_GET_SIZE(args[1]);
    const long code = PyLong_AsLong(args[2]), device = PyLong_AsLong(args[3]);
    at::ScalarType type;
    if (PyErr_Occurred()) return nullptr;
    if (!scalar_type(code, &type) || n < 0) {
        PyErr_SetString(PyExc_ValueError, "buffers: unknown dtype code or negative count");
        return nullptr;
    }
    std::vector<int64_t> shape((size_t)nd);
    for (Py_ssize_t d = 0; d < nd; ++d) shape[(size_t)d] = PyLong_AsLongLong(PyTuple_GET_ITEM(args[1], d));
    if (PyErr_Occurred()) return nullptr;
    PyObject* list = PyList_New(n);
    if (!list) return nullptr;
    try {
        const auto opts = at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject* o = THPVariable_Wrap(at::empty(shape, opts));
            if (!o) {
                Py_DECREF(list);
                return nullptr;
            }
            PyList_SET_ITEM(list, i, o);
        }
        return list;
    } catch (const c10::OutOfMemoryError& e) {
        Py_DECREF(list);
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* oom = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(oom ? oom : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(oom);
        Py_XDECREF(torch);
        return nullptr;
    } catch (const std::exception& e) {
        Py_DECREF(list);
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// ---- whole calls -------------------------------------------------------------------

using LinearFn = int (*)(int, int, int64_t, int64_t, int64_t, const void* const*, const void* const*, const void* const*,
                         const void* const*, int, int, void* const*, void* const*, void*);
using GluFn = int (*)(int, int64_t, int64_t, int64_t, int64_t, const void*, const void* const*, const void* const*,
                      const void* const*, const void*, int, void* const*, int, void*, void*);
using ClipFn = int (*)(int, const int32_t*, const int64_t*, const void* const*, const uint8_t*, float, void* const*, void*,
                       float*, void*);
LinearFn linear_fn = nullptr;
GluFn glu_fn = nullptr;
ClipFn clip_fn = nullptr;
decltype(&rtp_tp_cross_entropy) loss_fn = nullptr;
decltype(&rtp_tp_cross_entropy_train) loss_train_fn = nullptr;
decltype(&rtp_tp_cross_entropy_workspace) loss_workspace_fn = nullptr;
decltype(&rtp_adamw_step) adamw_fn = nullptr;

// bind(addresses of rtp_tp_linear, rtp_tp_glu, rtp_clip_grad_norm, rtp_tp_cross_entropy,
// rtp_tp_cross_entropy_train, rtp_tp_cross_entropy_workspace, rtp_adamw_step)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 7) {
        PyErr_SetString(PyExc_TypeError, "bind(linear, glu, clip, loss, loss_train, loss_workspace, adamw)");
        return nullptr;
    }
    uintptr_t at[7];
    for (int i = 0; i < 7; ++i) at[i] = (uintptr_t)PyLong_AsUnsignedLongLong(args[i]);
    if (PyErr_Occurred()) return nullptr;
    linear_fn = reinterpret_cast<LinearFn>(at[0]);
    glu_fn = reinterpret_cast<GluFn>(at[1]);
    clip_fn = reinterpret_cast<ClipFn>(at[2]);
    loss_fn = reinterpret_cast<decltype(loss_fn)>(at[3]);
    loss_train_fn = reinterpret_cast<decltype(loss_train_fn)>(at[4]);
    loss_workspace_fn = reinterpret_cast<decltype(loss_workspace_fn)>(at[5]);
    adamw_fn = reinterpret_cast<decltype(adamw_fn)>(at[6]);
    Py_RETURN_NONE;
}

constexpr int MAX_RANKS = 8;

bool fits(const at::Tensor& t, at::IntArrayRef shape, long device)
{
    return t.scalar_type() == at::kBFloat16 && t.sizes() == shape && placed(t, device);
}

// The addresses of the n bf16 tensors of a list (or of one tensor, n = 1).
bool addresses(PyObject* o, Py_ssize_t n, at::IntArrayRef shape, long device, const void** out)
{
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (n != 1 || !fits(t, shape, device)) return false;
        out[0] = t.data_ptr();
        return true;
    }
    if (!PyList_Check(o) || PyList_GET_SIZE(o) != n) return false;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject* e = PyList_GET_ITEM(o, i);
        if (!THPVariable_Check(e)) return false;
        const at::Tensor& t = THPVariable_Unpack(e);
        if (!fits(t, shape, device)) return false;
        out[i] = t.data_ptr();
    }
    return true;
}

// Shape of a matrix, or of the first one of a list.
bool matrix(PyObject* o, int64_t* rows, int64_t* cols, long device)
{
    if (PyList_Check(o) && PyList_GET_SIZE(o) > 0) o = PyList_GET_ITEM(o, 0);
    if (!THPVariable_Check(o)) return false;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 2 || !t.is_cuda() || t.get_device() != device) return false;
    *rows = t.size(0);
    *cols = t.size(1);
    return true;
}

at::TensorOptions bf16_on(long device)
{
    return at::TensorOptions().dtype(at::kBFloat16).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
}

// linear(X, W, row, bias, residual, act, device, stream): rtp_tp_linear with new bf16
// outputs. Returns their list; a status; or None when an argument is not what the
// call takes (the Python code then says which).
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 8 || !linear_fn) {
        PyErr_SetString(PyExc_TypeError, "linear(X, W, row, bias, residual, act, device, stream)");
        return nullptr;
    }
    const bool row = args[2] == Py_True;
    const long act = PyLong_AsLong(args[5]), device = PyLong_AsLong(args[6]);
    const unsigned long long stream = PyLong_AsUnsignedLongLong(args[7]);
    if (PyErr_Occurred()) return nullptr;
    if (!PyList_Check(args[1])) Py_RETURN_NONE;
    const Py_ssize_t P = PyList_GET_SIZE(args[1]);
    int64_t M, Kx, Kp, Np;
    if (P < 1 || P > MAX_RANKS || !matrix(args[0], &M, &Kx, device) || !matrix(args[1], &Kp, &Np, device)) Py_RETURN_NONE;
    const Py_ssize_t outs = row ? 1 : P;
    const void *x[MAX_RANKS], *w[MAX_RANKS], *b[MAX_RANKS], *r[MAX_RANKS];
    void* o[MAX_RANKS];
    const bool has_b = args[3] != Py_None, has_r = args[4] != Py_None;
    if (!addresses(args[0], row ? P : 1, {M, Kp}, device, x) || !addresses(args[1], P, {Kp, Np}, device, w) ||
        (has_b && !addresses(args[3], outs, {Np}, device, b)) || (has_r && !addresses(args[4], outs, {M, Np}, device, r)))
        Py_RETURN_NONE;
    PyObject* list = PyList_New(outs);
    if (!list) return nullptr;
    try {
        for (Py_ssize_t i = 0; i < outs; ++i) {
            at::Tensor t = at::empty({M, Np}, bf16_on(device));
            o[i] = t.data_ptr();
            PyObject* e = THPVariable_Wrap(std::move(t));
            if (!e) {
                Py_DECREF(list);
                return nullptr;
            }
            PyList_SET_ITEM(list, i, e);
        }
    } catch (const std::exception&) {  // out of memory: the Python code raises it
        Py_DECREF(list);
        Py_RETURN_NONE;
    }
    const int rc = linear_fn(row ? 1 : 0, (int)P, M, row ? Kp * P : Kp, row ? Np : Np * P, x, w, has_b ? b : nullptr,
                             has_r ? r : nullptr, (int)act, 1, nullptr, o, reinterpret_cast<void*>((uintptr_t)stream));
    if (rc == 0) return list;
    Py_DECREF(list);
    return PyLong_FromLong(rc);
}

// glu(X, Ag, Au, B, residual, act, device, stream): rtp_tp_glu with a new bf16 Z and
// scratch for Y; returns as linear() does.
PyObject* glu(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 8 || !glu_fn) {
        PyErr_SetString(PyExc_TypeError, "glu(X, Ag, Au, B, residual, act, device, stream)");
        return nullptr;
    }
    const long act = PyLong_AsLong(args[5]), device = PyLong_AsLong(args[6]);
    const unsigned long long stream = PyLong_AsUnsignedLongLong(args[7]);
    if (PyErr_Occurred()) return nullptr;
    if (!PyList_Check(args[1])) Py_RETURN_NONE;
    const Py_ssize_t P = PyList_GET_SIZE(args[1]);
    int64_t M, K, Kg, Fp, Fb, N;
    if (P < 1 || P > MAX_RANKS || !matrix(args[0], &M, &K, device) || !matrix(args[1], &Kg, &Fp, device) ||
        !matrix(args[3], &Fb, &N, device))
        Py_RETURN_NONE;
    const void *x[1], *g[MAX_RANKS], *u[MAX_RANKS], *b[MAX_RANKS], *r[1] = {nullptr};
    if (!addresses(args[0], 1, {M, K}, device, x) || !addresses(args[1], P, {K, Fp}, device, g) ||
        !addresses(args[2], P, {K, Fp}, device, u) || !addresses(args[3], P, {Fp, N}, device, b) ||
        (args[4] != Py_None && !addresses(args[4], 1, {M, N}, device, r)))
        Py_RETURN_NONE;
    at::Tensor Y, Z;
    try {
        Y = at::empty({P, M, Fp}, bf16_on(device));
        Z = at::empty({M, N}, bf16_on(device));
    } catch (const std::exception&) {
        Py_RETURN_NONE;
    }
    void* y[MAX_RANKS];
    for (Py_ssize_t i = 0; i < P; ++i) y[i] = static_cast<char*>(Y.data_ptr()) + i * M * Fp * 2;
    const int rc = glu_fn((int)P, M, K, Fp * P, N, x[0], g, u, b, r[0], (int)act, y, 1, Z.data_ptr(),
                          reinterpret_cast<void*>((uintptr_t)stream));
    return rc == 0 ? THPVariable_Wrap(std::move(Z)) : PyLong_FromLong(rc);
}

// Whether the tables of a group still say what its tensors are: a tensor's storage
// can be replaced under it, and the one tabulated be freed.
bool same(PyObject* list, const int32_t* dtypes, const int64_t* numels, const void* const* at, long device)
{
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(list); ++i) {
        PyObject* o = PyList_GET_ITEM(list, i);
        if (!THPVariable_Check(o)) return false;
        const at::Tensor& t = THPVariable_Unpack(o);
        at::ScalarType want;
        if (!scalar_type(dtypes[i], &want) || t.scalar_type() != want || t.numel() != numels[i]) return false;
        if (numels[i] > 0 && (!placed(t, device) || t.data_ptr() != at[i])) return false;
    }
    return true;
}

// unchanged(n, dtypes, numels, grads, tensors, device) -> bool
PyObject* unchanged(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 6 || !PyList_Check(args[4])) {
        PyErr_SetString(PyExc_TypeError, "unchanged(n, dtypes, numels, grads, tensors, device)");
        return nullptr;
    }
    const long n = PyLong_AsLong(args[0]), device = PyLong_AsLong(args[5]);
    unsigned long long at[3];
    for (int i = 0; i < 3; ++i) at[i] = PyLong_AsUnsignedLongLong(args[1 + i]);
    if (PyErr_Occurred()) return nullptr;
    auto p = [&](int i) { return reinterpret_cast<void*>((uintptr_t)at[i]); };
    return PyBool_FromLong(PyList_GET_SIZE(args[4]) == n &&
                           same(args[4], static_cast<const int32_t*>(p(0)), static_cast<const int64_t*>(p(1)),
                                static_cast<const void* const*>(p(2)), device));
}

// clip(n, dtypes, numels, grads, counted, workspace, max_norm, out, tensors, device,
// stream): rtp_clip_grad_norm on a group's tables (addresses) with a new norm tensor;
// out: None (in place) or a list like `tensors`. Returns as linear() does, None also
// where the tables are not of `tensors` any more.
PyObject* clip(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 11 || !clip_fn || !PyList_Check(args[8])) {
        PyErr_SetString(PyExc_TypeError,
                        "clip(n, dtypes, numels, grads, counted, workspace, max_norm, out, tensors, device, stream)");
        return nullptr;
    }
    const long n = PyLong_AsLong(args[0]), device = PyLong_AsLong(args[9]);
    unsigned long long at[5], stream = PyLong_AsUnsignedLongLong(args[10]);
    for (int i = 0; i < 5; ++i) at[i] = PyLong_AsUnsignedLongLong(args[1 + i]);
    const double max_norm = PyFloat_AsDouble(args[6]);
    if (PyErr_Occurred()) return nullptr;
    if (n < 0 || PyList_GET_SIZE(args[8]) != n) Py_RETURN_NONE;
    auto p = [&](int i) { return reinterpret_cast<void*>((uintptr_t)at[i]); };
    try {
        if (!same(args[8], static_cast<const int32_t*>(p(0)), static_cast<const int64_t*>(p(1)),
                  static_cast<const void* const*>(p(2)), device))
            Py_RETURN_NONE;
        std::vector<void*> out;
        if (args[7] != Py_None) {
            if (!PyList_Check(args[7]) || PyList_GET_SIZE(args[7]) != n) Py_RETURN_NONE;
            out.resize((size_t)n + 1);  // never without storage: a NULL table means in place
            for (Py_ssize_t i = 0; i < n; ++i) {
                PyObject *a = PyList_GET_ITEM(args[7], i), *b = PyList_GET_ITEM(args[8], i);
                if (!THPVariable_Check(a) || !THPVariable_Check(b)) Py_RETURN_NONE;
                const at::Tensor &t = THPVariable_Unpack(a), &r = THPVariable_Unpack(b);
                if (t.scalar_type() != r.scalar_type() || t.sizes() != r.sizes() || !placed(t, device)) Py_RETURN_NONE;
                out[(size_t)i] = t.data_ptr();
            }
        }
        at::Tensor norm = at::empty(at::IntArrayRef{}, at::TensorOptions().dtype(at::kFloat).device(
                                                           c10::Device(c10::kCUDA, (c10::DeviceIndex)device)));
        const int rc = clip_fn((int)n, static_cast<const int32_t*>(p(0)), static_cast<const int64_t*>(p(1)),
                               static_cast<const void* const*>(p(2)), static_cast<const uint8_t*>(p(3)), (float)max_norm,
                               out.empty() ? nullptr : out.data(), p(4), norm.data_ptr<float>(),
                               reinterpret_cast<void*>((uintptr_t)stream));
        return rc == 0 ? THPVariable_Wrap(std::move(norm)) : PyLong_FromLong(rc);
    } catch (const std::exception&) {
        Py_RETURN_NONE;
    }
}

// ---- losses and the AdamW step -------------------------------------------------------

at::TensorOptions on(at::ScalarType type, long device)
{
    return at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
}

// What both loss calls take: X, W, targets.
struct LossArguments {
    int P;
    int64_t M, K, Vp;
    const void *x[1], *w[MAX_RANKS], *targets;
    int wide;
};
bool loss_arguments(PyObject* const* args, long device, LossArguments* a)
{
    if (!PyList_Check(args[1]) || !THPVariable_Check(args[2])) return false;
    const Py_ssize_t P = PyList_GET_SIZE(args[1]);
    int64_t Kw;
    if (P < 1 || P > MAX_RANKS || PyList_Check(args[0]) || !matrix(args[0], &a->M, &a->K, device) ||
        !matrix(args[1], &Kw, &a->Vp, device))
        return false;
    const at::Tensor& t = THPVariable_Unpack(args[2]);
    if ((t.scalar_type() != at::kLong && t.scalar_type() != at::kInt) || t.sizes() != at::IntArrayRef{a->M} || !placed(t, device) ||
        !addresses(args[0], 1, {a->M, a->K}, device, a->x) || !addresses(args[1], P, {a->K, a->Vp}, device, a->w))
        return false;
    a->P = (int)P;
    a->targets = t.data_ptr();
    a->wide = t.scalar_type() == at::kLong;
    return true;
}

// loss(X, W, targets, vocab, ignore, device, stream): rtp_tp_cross_entropy with new
// outputs and workspace, vocab < 0: all columns. Returns (loss, lse), or as linear() does.
PyObject* loss(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 7 || !loss_fn) {
        PyErr_SetString(PyExc_TypeError, "loss(X, W, targets, vocab, ignore, device, stream)");
        return nullptr;
    }
    const long long vocab = PyLong_AsLongLong(args[3]), ignore = PyLong_AsLongLong(args[4]);
    const long device = PyLong_AsLong(args[5]);
    const unsigned long long stream = PyLong_AsUnsignedLongLong(args[6]);
    if (PyErr_Occurred()) return nullptr;
    LossArguments a;
    if (!loss_arguments(args, device, &a)) Py_RETURN_NONE;
    const int64_t V = a.Vp * a.P;
    int64_t bytes = 0;
    int rc = loss_workspace_fn(a.P, a.M, a.K, V, 0, 0, RTP_F32, &bytes);
    if (rc) return PyLong_FromLong(rc);
    at::Tensor l, s, ws;
    try {
        l = at::empty({a.M}, on(at::kFloat, device));
        s = at::empty({a.M}, on(at::kFloat, device));
        ws = at::empty({bytes}, on(at::kByte, device));
    } catch (const std::exception&) {  // out of memory: the Python code raises it
        Py_RETURN_NONE;
    }
    rc = loss_fn(a.P, a.M, a.K, V, vocab < 0 ? V : vocab, a.x[0], a.w, a.wide, a.targets, ignore, ws.data_ptr(), bytes,
                 l.data_ptr<float>(), s.data_ptr<float>(), reinterpret_cast<void*>((uintptr_t)stream));
    if (rc) return PyLong_FromLong(rc);
    return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(l)), THPVariable_Wrap(std::move(s)));
}

// loss_train(X, W, targets, weights, vocab, ignore, mean, scale, device, stream):
// rtp_tp_cross_entropy_train with new bf16 gradients. Returns (total, loss, dX, dW).
PyObject* loss_train(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 10 || !loss_train_fn) {
        PyErr_SetString(PyExc_TypeError, "loss_train(X, W, targets, weights, vocab, ignore, mean, scale, device, stream)");
        return nullptr;
    }
    const long long vocab = PyLong_AsLongLong(args[4]), ignore = PyLong_AsLongLong(args[5]);
    const bool mean = args[6] == Py_True;
    const double scale = PyFloat_AsDouble(args[7]);
    const long device = PyLong_AsLong(args[8]);
    const unsigned long long stream = PyLong_AsUnsignedLongLong(args[9]);
    if (PyErr_Occurred()) return nullptr;
    LossArguments a;
    if (!loss_arguments(args, device, &a)) Py_RETURN_NONE;
    const float* weights = nullptr;
    if (args[3] != Py_None) {
        if (!THPVariable_Check(args[3])) Py_RETURN_NONE;
        const at::Tensor& t = THPVariable_Unpack(args[3]);
        if (t.scalar_type() != at::kFloat || t.sizes() != at::IntArrayRef{a.M} || !placed(t, device)) Py_RETURN_NONE;
        weights = static_cast<const float*>(t.data_ptr());
    }
    const int64_t V = a.Vp * a.P;
    int64_t bytes = 0;
    int rc = loss_workspace_fn(a.P, a.M, a.K, V, 0, 1, RTP_BF16, &bytes);
    if (rc) return PyLong_FromLong(rc);
    at::Tensor total, l, dx, ws, dw[MAX_RANKS];
    void* dwp[MAX_RANKS];
    try {
        total = at::empty(at::IntArrayRef{}, on(at::kFloat, device));
        l = at::empty({a.M}, on(at::kFloat, device));
        dx = at::empty({a.M, a.K}, bf16_on(device));
        for (int i = 0; i < a.P; ++i) {
            dw[i] = at::empty({a.K, a.Vp}, bf16_on(device));
            dwp[i] = dw[i].data_ptr();
        }
        ws = at::empty({bytes}, on(at::kByte, device));
    } catch (const std::exception&) {
        Py_RETURN_NONE;
    }
    rc = loss_train_fn(a.P, a.M, a.K, V, vocab < 0 ? V : vocab, a.x[0], a.w, a.wide, a.targets, ignore, weights, mean, (float)scale, 0,
                       ws.data_ptr(), bytes, total.data_ptr<float>(), l.data_ptr<float>(), RTP_BF16, dx.data_ptr(), RTP_BF16, dwp,
                       0, reinterpret_cast<void*>((uintptr_t)stream));
    if (rc) return PyLong_FromLong(rc);
    PyObject* list = PyList_New(a.P);
    if (!list) return nullptr;
    for (int i = 0; i < a.P; ++i) {
        PyObject* e = THPVariable_Wrap(std::move(dw[i]));
        if (!e) {
            Py_DECREF(list);
            return nullptr;
        }
        PyList_SET_ITEM(list, i, e);
    }
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(std::move(total)), THPVariable_Wrap(std::move(l)),
                         THPVariable_Wrap(std::move(dx)), list);
}

// A float32 scalar on the device: its address, or NULL.
const float* scalar_on(PyObject* o, long device)
{
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != at::kFloat || t.numel() != 1 || t.get_device() != device) return nullptr;
    return static_cast<const float*>(t.data_ptr());
}

// adamw(table, n, params, masters, grads, bits, lr, eps, norm, max_norm, seed, clock,
// device, stream): rtp_adamw_step on a group's table (an address), which is brought up to
// the tensors as they are. lr: a number or a scalar tensor; norm: None or a scalar tensor.
// Returns True; a status; or None when a tensor is not what the group was built over.
PyObject* adamw(PyObject*, PyObject* const* args, Py_ssize_t nargs)
{
    if (nargs != 14 || !adamw_fn || !PyList_Check(args[2]) || !PyList_Check(args[3]) || !PyList_Check(args[4])) {
        PyErr_SetString(PyExc_TypeError,
                        "adamw(table, n, params, masters, grads, bits, lr, eps, norm, max_norm, seed, clock, device, stream)");
        return nullptr;
    }
    auto* table = reinterpret_cast<rtp_adamw_tensor*>((uintptr_t)PyLong_AsUnsignedLongLong(args[0]));
    const long n = PyLong_AsLong(args[1]), bits = PyLong_AsLong(args[5]), device = PyLong_AsLong(args[12]);
    const double eps = PyFloat_AsDouble(args[7]), max_norm = PyFloat_AsDouble(args[9]);
    const unsigned long long seed = PyLong_AsUnsignedLongLong(args[10]), clock = PyLong_AsUnsignedLongLong(args[11]),
                             stream = PyLong_AsUnsignedLongLong(args[13]);
    if (PyErr_Occurred()) return nullptr;
    const float *lr_at = nullptr, *norm = nullptr;
    double lr = 0.0;
    if (PyFloat_Check(args[6])) lr = PyFloat_AS_DOUBLE(args[6]);
    else if (!(lr_at = scalar_on(args[6], device))) Py_RETURN_NONE;
    if (args[8] != Py_None && !(norm = scalar_on(args[8], device))) Py_RETURN_NONE;
    for (int k = 2; k < 5; ++k)
        if (PyList_GET_SIZE(args[k]) != n) Py_RETURN_NONE;
    for (long i = 0; i < n; ++i) {
        PyObject *po = PyList_GET_ITEM(args[2], i), *mo = PyList_GET_ITEM(args[3], i), *go = PyList_GET_ITEM(args[4], i);
        if (!THPVariable_Check(po) || !THPVariable_Check(go) || (mo != Py_None && !THPVariable_Check(mo))) Py_RETURN_NONE;
        const at::Tensor &p = THPVariable_Unpack(po), &g = THPVariable_Unpack(go);
        rtp_adamw_tensor& t = table[i];
        at::ScalarType want;
        if (!scalar_type(t.param_dtype, &want) || p.scalar_type() != want || p.numel() != t.numel || !placed(p, device)) Py_RETURN_NONE;
        if ((g.scalar_type() != at::kFloat && g.scalar_type() != at::kBFloat16) || g.sizes() != p.sizes() || !placed(g, device))
            Py_RETURN_NONE;
        void* master = nullptr;
        if (mo != Py_None) {
            const at::Tensor& m = THPVariable_Unpack(mo);
            if (m.scalar_type() != at::kFloat || want != at::kBFloat16 || m.sizes() != p.sizes() || !placed(m, device)) Py_RETURN_NONE;
            master = m.data_ptr();
        }
        t.param = p.data_ptr();
        t.master = static_cast<float*>(master);
        t.grad = g.data_ptr();
        t.grad_dtype = g.scalar_type() == at::kFloat ? RTP_F32 : RTP_BF16;
    }
    const int rc = adamw_fn((int)n, table, (int)bits, (float)lr, lr_at, (float)eps, norm, (float)max_norm, (uint32_t)seed,
                            reinterpret_cast<void*>((uintptr_t)clock), reinterpret_cast<void*>((uintptr_t)stream));
    if (rc) return PyLong_FromLong(rc);
    Py_RETURN_TRUE;
}

// A method of the module. No C++ exception leaves it: tensors that torch itself wraps,
// or that have no storage, raise from the very calls that ask for their addresses.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* method(PyObject* self, PyObject* const* args, Py_ssize_t nargs) noexcept
{
    try {
        return F(self, args, nargs);
    } catch (python_error& e) {
        e.restore();
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::bad_alloc&) {
        PyErr_NoMemory();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "an unknown C++ exception");
    }
    return nullptr;
}
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef entry(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(method<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {entry<bind>("bind"),       entry<table>("table"),         entry<like>("like"),
                         entry<buffers>("buffers"), entry<linear>("linear"),       entry<glu>("glu"),
                         entry<clip>("clip"),       entry<unchanged>("unchanged"), entry<loss>("loss"),
                         entry<loss_train>("loss_train"), entry<adamw>("adamw"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_table", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__table() { return PyModule_Create(&module); }
