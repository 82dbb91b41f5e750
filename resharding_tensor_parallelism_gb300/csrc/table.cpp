// Python extension of the binding: allocates lists of buffers, and checks a list of torch tensors against the
// type, shape and device that a call will touch, and returns their addresses as
// one table of 64-bit pointers. The same checks as the binding's Python loop, at
// about 20 ns a tensor instead of 500: a call on 8 ranks passes 20 to 60
// tensors, and a decoded token's product takes the GPU about as long as that loop.
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <vector>

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
    try {
        std::vector<uint64_t> out((size_t)n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject* o = PyList_GET_ITEM(args[0], i);
            if (!THPVariable_Check(o)) return PyLong_FromSsize_t(i);
            const at::Tensor& t = THPVariable_Unpack(o);
            if (t.scalar_type() != want || t.sizes() != sizes || !placed(t, device)) return PyLong_FromSsize_t(i);
            out[(size_t)i] = (uint64_t)(uintptr_t)t.data_ptr();
        }
        return pointers(out);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
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
    try {
        std::vector<uint64_t> out((size_t)n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject *a = PyList_GET_ITEM(args[0], i), *b = PyList_GET_ITEM(args[1], i);
            if (!THPVariable_Check(a) || !THPVariable_Check(b)) return PyLong_FromSsize_t(i);
            const at::Tensor &t = THPVariable_Unpack(a), &r = THPVariable_Unpack(b);
            if (t.scalar_type() != r.scalar_type() || t.sizes() != r.sizes() || !placed(t, device)) return PyLong_FromSsize_t(i);
            out[(size_t)i] = (uint64_t)(uintptr_t)t.data_ptr();
        }
        return pointers(out);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
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

PyMethodDef methods[] = {
    {"buffers", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(buffers)), METH_FASTCALL, nullptr},
    {"table", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(table)), METH_FASTCALL, nullptr},
    {"like", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(like)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_table", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__table() { return PyModule_Create(&module); }
