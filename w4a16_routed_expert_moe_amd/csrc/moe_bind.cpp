// moe_bind.cpp -- the binding's check of one tensor argument, natively.
//
// at(dev, t, name, dtype, numel, optional=False): the address of t if it is a
// contiguous tensor on device dev with that type and at least numel elements.
// Every other argument (None, a subclass, whatever fails a check) goes to the
// Python function given to set_checked, which decides and words the error.  A
// call checks up to 17 tensors, and a decode step's calls are bound by the
// host: 0.05 us a tensor here against 0.3 for the same checks in Python (a
// one-row projection 6.2 -> 5.2 us, the router's loss and gradient 14.1 -> 11.1).
// built_for: the Python and torch of the headers that this was compiled with
// (the build gives MOE_BUILT_FOR); only there are the offsets read here right.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

PyObject *checked = nullptr;

PyObject *at(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n < 5) {
        PyErr_SetString(PyExc_TypeError, "at(dev, t, name, dtype, numel, optional=False)");
        return nullptr;
    }
    if (THPVariable_CheckExact(args[1]) && THPDtype_Check(args[3])) {
        const at::Tensor &t = THPVariable_Unpack(args[1]);
        const long dev = PyLong_AsLong(args[0]);
        const long long numel = PyLong_AsLongLong(args[4]);
        if (PyErr_Occurred()) return nullptr;
        try {
            if (t.layout() == c10::kStrided && t.get_device() == dev &&
                t.scalar_type() == ((THPDtype *)args[3])->scalar_type && t.is_contiguous() && t.numel() >= numel)
                // the address to write through, as Tensor.data_ptr() gives it:
                // a copy-on-write tensor gets memory of its own first
                return PyLong_FromVoidPtr(t.mutable_data_ptr());
        } catch (const std::exception &) {  // a tensor without memory (one that torch.func wraps, say)
        }
    }
    if (!checked) {
        PyErr_SetString(PyExc_RuntimeError, "set_checked has not been called");
        return nullptr;
    }
    return PyObject_Vectorcall(checked, args, n, nullptr);
}

PyObject *set_checked(PyObject *, PyObject *fn) {
    Py_INCREF(fn);
    Py_XSETREF(checked, fn);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"at", (PyCFunction)(void (*)(void))at, METH_FASTCALL, "address of a checked tensor"},
                         {"set_checked", set_checked, METH_O, "the function for arguments that at does not pass"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "native argument checks", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", MOE_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
