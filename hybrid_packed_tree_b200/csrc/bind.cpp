// bind.cpp -- the argument check of the Python binding, in C++.
//
// A decode step makes several calls per layer, each with about ten tensors: shape, dtype,
// device and layout asked for one by one in Python cost 0.4 us a tensor, more than the launch.
//
//   arg(tensor, name, shape, dtype, device) -> the data pointer as an int
//   opt(tensor or None, ...) the same, None for None
//   on_refusal(function): called with the same arguments when the tensor is not contiguous, of exactly
//     this shape and dtype, on this CUDA device; it raises the error that says which.
#include <Python.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

PyObject *g_refuse = nullptr;

bool fits(PyObject *t, PyObject *shape, PyObject *dtype, PyObject *device, const void **ptr)
{
    if (!THPVariable_Check(t) || !PyTuple_Check(shape) || !THPDtype_Check(dtype)) return false;
    const at::Tensor &x = THPVariable_Unpack(t);
    const long dev = PyLong_AsLong(device);
    if (dev < 0 || !x.defined() || x.layout() != at::kStrided || !x.is_cuda() || x.get_device() != dev ||
        x.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type)
        return false;
    const auto sizes = x.sizes();
    if (PyTuple_GET_SIZE(shape) != (Py_ssize_t)sizes.size()) return false;
    for (size_t i = 0; i < sizes.size(); ++i)
        if (PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i)) != sizes[i]) return false;
    if (!x.is_contiguous()) return false;
    *ptr = x.data_ptr();
    return true;
}

PyObject *check(PyObject *const *args, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "(tensor, name, shape, dtype, device) expected");
        return nullptr;
    }
    try {
        const void *ptr = nullptr;
        if (fits(args[0], args[2], args[3], args[4], &ptr)) return PyLong_FromUnsignedLongLong((unsigned long long)(uintptr_t)ptr);
    } catch (const std::exception &e) {        // a tensor without storage and the like
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    if (PyErr_Occurred()) return nullptr;
    if (!g_refuse) {
        PyErr_SetString(PyExc_TypeError, "argument refused");
        return nullptr;
    }
    return PyObject_Vectorcall(g_refuse, args, 5, nullptr);
}

PyObject *arg(PyObject *, PyObject *const *args, Py_ssize_t n) { return check(args, n); }

PyObject *opt(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n >= 1 && args[0] == Py_None) Py_RETURN_NONE;
    return check(args, n);
}

PyObject *on_refusal(PyObject *, PyObject *f)
{
    Py_INCREF(f);
    Py_XSETREF(g_refuse, f);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"arg", (PyCFunction)(void (*)(void))arg, METH_FASTCALL, "The pointer of a tensor of this shape, dtype and device."},
    {"opt", (PyCFunction)(void (*)(void))opt, METH_FASTCALL, "arg, or None for None."},
    {"on_refusal", on_refusal, METH_O, "The function that raises for a tensor that does not fit."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind(void) { return PyModule_Create(&module); }
