// operands.cpp -- the checks that every call from Python makes of its operands, compiled: gemm_epi.py's _operand and
// _device_and_stream for the case where all is well.  Anything else is handed to the Python function of the same name, which
// decides and words the error, so there is one place that says what an operand has to be.
//
// A call from Python with six operands spends 2.5 us in the Python forms and 0.4 us in these, beside 1.2 us of ctypes and
// 2.1 us of the launch.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

namespace {

PyObject *slow_operand = nullptr, *slow_stream = nullptr;

bool have_python_forms() {
    if (slow_operand == nullptr) PyErr_SetString(PyExc_RuntimeError, "_operands: set_python_forms comes first");
    return slow_operand != nullptr;
}

// Whether obj is a tensor of this dtype, shape (a tuple) and device, contiguous.
bool fits(PyObject *obj, PyObject *dtype, PyObject *shape, PyObject *device) {
    if (!THPVariable_Check(obj) || !THPDtype_Check(dtype) || !PyTuple_CheckExact(shape) || !PyLong_CheckExact(device)) return false;
    const at::Tensor &t = THPVariable_Unpack(obj);
    if (t.layout() != at::kStrided || t.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type) return false;
    const auto sizes = t.sizes();
    const Py_ssize_t n = PyTuple_GET_SIZE(shape);
    if ((Py_ssize_t)sizes.size() != n) return false;
    for (Py_ssize_t i = 0; i < n; ++i) {
        PyObject *want = PyTuple_GET_ITEM(shape, i);
        if (!PyLong_CheckExact(want) || PyLong_AsLongLong(want) != sizes[i]) return false;
    }
    return t.is_contiguous() && (t.is_cpu() || t.is_cuda()) && PyLong_AsLong(device) == (t.is_cuda() ? t.device().index() : -1);
}

// operand(t, name, dtype, shape, device[, optional]): the address, as gemm_epi.py's.
PyObject *operand(PyObject *, PyObject *const *args, Py_ssize_t nargs) {
    if (nargs == 6 && args[0] == Py_None && args[5] == Py_True) Py_RETURN_NONE;
    if ((nargs == 5 || nargs == 6) && args[0] != Py_None) {
        try {
            // (mutable: a call may write there, and a copy-on-write tensor gets memory of its own first)
            if (fits(args[0], args[2], args[3], args[4])) return PyLong_FromVoidPtr(THPVariable_Unpack(args[0]).mutable_data_ptr());
        } catch (const std::exception &) {            // a tensor without memory of its own: the Python form's to say
        }
        PyErr_Clear();                                // (a size beyond 64 bits)
    }
    return have_python_forms() ? PyObject_Vectorcall(slow_operand, args, (size_t)nargs, nullptr) : nullptr;
}

// device_and_stream(stream): (current device, its current stream's handle) when stream is None.
PyObject *device_and_stream(PyObject *, PyObject *stream) {
    if (stream == Py_None) {
        try {
            const auto s = c10::cuda::getCurrentCUDAStream();
            return Py_BuildValue("(iK)", (int)s.device_index(), (unsigned long long)reinterpret_cast<uintptr_t>(s.stream()));
        } catch (const std::exception &) {            // no device: as torch reports it
        }
    }
    return have_python_forms() ? PyObject_CallOneArg(slow_stream, stream) : nullptr;
}

// Whether f is one of the two functions here, which would hand on to itself without end.
bool compiled_form(PyObject *f) {
    if (!PyCFunction_Check(f)) return false;
    const PyCFunction c = PyCFunction_GetFunction(f);
    return c == device_and_stream || c == reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(operand));
}

PyObject *set_python_forms(PyObject *, PyObject *args) {
    PyObject *a, *b;
    if (!PyArg_ParseTuple(args, "OO", &a, &b)) return nullptr;
    if (!PyCallable_Check(a) || !PyCallable_Check(b) || compiled_form(a) || compiled_form(b)) {
        PyErr_SetString(PyExc_TypeError, "set_python_forms: the Python forms of operand and device_and_stream");
        return nullptr;
    }
    Py_INCREF(a);
    Py_INCREF(b);
    Py_XSETREF(slow_operand, a);
    Py_XSETREF(slow_stream, b);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"operand", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(operand)), METH_FASTCALL, nullptr},
    {"device_and_stream", device_and_stream, METH_O, nullptr},
    {"set_python_forms", set_python_forms, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operands", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: torch's version and Python's, which have to be the running ones before anything here is called (tensors are read by
// the layout that torch's headers gave them).
PyMODINIT_FUNC PyInit__operands() {
    PyObject *m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
