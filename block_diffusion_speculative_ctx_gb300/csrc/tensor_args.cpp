// Checks of tensor arguments for the Python operators (ops.py), and the versions of the tensors that they write, as a CPython
// extension: type, size, device and layout of a tensor are read from the tensor itself instead of attribute by attribute through Python (some 0.4 us a tensor; a call
// takes up to twelve, and a small call is as long as its host side).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

namespace {

const at::Tensor* tensor(PyObject* o) {
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    PyErr_Format(PyExc_ValueError, "a tensor is expected, not %R", Py_TYPE(o));
    return nullptr;
}

// "<name> must be <what> on cuda:<dev>, not <dtype> <shape> on <device>"
PyObject* refuse(PyObject* name, PyObject* what, long dev, PyObject* t) {
    PyObject *dtype = PyObject_GetAttrString(t, "dtype"), *shape = PyObject_GetAttrString(t, "shape"),
             *device = PyObject_GetAttrString(t, "device"), *list = shape ? PySequence_List(shape) : nullptr;
    if (what && dtype && list && device)
        PyErr_Format(PyExc_ValueError, "%U must be %U on cuda:%ld, not %S %S on %S", name, what, dev, dtype, list, device);
    Py_XDECREF(what);
    Py_XDECREF(dtype);
    Py_XDECREF(shape);
    Py_XDECREF(device);
    Py_XDECREF(list);
    return nullptr;
}

template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
}

bool args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return false;
}

bool of_type(const at::Tensor& t, PyObject* dtype) {
    return THPDtype_Check(dtype) && reinterpret_cast<THPDtype*>(dtype)->scalar_type == t.scalar_type();
}

// flat(name, t, dtype, n, dev): address of a contiguous tensor of n elements
PyObject* flat(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!args(na, 5)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor* t = tensor(a[1]);
        const long long n = PyLong_AsLongLong(a[3]);
        const long dev = PyLong_AsLong(a[4]);
        if (!t || PyErr_Occurred()) return nullptr;
        if (!of_type(*t, a[2]) || t->numel() != n || t->get_device() != dev || !t->is_contiguous())
            return refuse(a[0], PyUnicode_FromFormat("a contiguous %S tensor of %lld elements", a[2], n), dev, a[1]);
        return PyLong_FromVoidPtr(t->data_ptr());
    });
}

// mat(name, t, dtype, rows, cols or None, dev): row stride, in elements, of a row-major matrix
PyObject* mat(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!args(na, 6)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor* t = tensor(a[1]);
        const long long rows = PyLong_AsLongLong(a[3]), cols = a[4] == Py_None ? -1 : PyLong_AsLongLong(a[4]);
        const long dev = PyLong_AsLong(a[5]);
        if (!t || PyErr_Occurred()) return nullptr;
        if (!of_type(*t, a[2]) || t->dim() != 2 || t->get_device() != dev || t->size(0) != rows || (cols >= 0 && t->size(1) != cols))
            return refuse(a[0],
                          cols < 0 ? PyUnicode_FromFormat("a %S matrix of %lld rows", a[2], rows)
                                   : PyUnicode_FromFormat("a %S [%lld, %lld]", a[2], rows, cols),
                          dev, a[1]);
        if (t->is_contiguous()) return PyLong_FromLongLong(t->size(1));
        const long long m = t->size(1), ld = rows <= 1 || m == 0 ? m : (long long)t->stride(0);
        if ((m > 1 && t->stride(1) != 1) || ld < m) return PyErr_Format(PyExc_ValueError, "%U must be row-major", a[0]);
        return PyLong_FromLongLong(ld);
    });
}

// rows3(name, t, dtype, rows, heads, hd, dev): row stride of a [rows, heads, hd] tensor whose rows are contiguous
PyObject* rows3(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!args(na, 7)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor* t = tensor(a[1]);
        const long long rows = PyLong_AsLongLong(a[3]), heads = PyLong_AsLongLong(a[4]), hd = PyLong_AsLongLong(a[5]);
        const long dev = PyLong_AsLong(a[6]);
        if (!t || PyErr_Occurred()) return nullptr;
        if (!of_type(*t, a[2]) || t->dim() != 3 || t->size(0) != rows || t->size(1) != heads || t->size(2) != hd ||
            t->get_device() != dev)
            return refuse(a[0], PyUnicode_FromFormat("a %S [%lld, %lld, %lld]", a[2], rows, heads, hd), dev, a[1]);
        if (t->is_contiguous()) return PyLong_FromLongLong(heads * hd);
        if ((hd > 1 && t->stride(2) != 1) || (heads > 1 && t->stride(1) != hd))
            return PyErr_Format(PyExc_ValueError, "%U: the heads of a row must be contiguous", a[0]);
        return PyLong_FromLongLong(rows > 1 ? (long long)t->stride(0) : heads * hd);
    });
}

// written(t, ...): the tensors (or None) have been written to: their versions rise, so that a backward pass that saved one of
// them says so
PyObject* written(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        for (Py_ssize_t i = 0; i < na; ++i) {
            if (a[i] == Py_None) continue;
            const at::Tensor* t = tensor(a[i]);
            if (!t) return nullptr;
            if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
        }
        Py_RETURN_NONE;
    });
}

PyMethodDef methods[] = {{"flat", (PyCFunction)(void (*)(void))flat, METH_FASTCALL, nullptr},
                         {"mat", (PyCFunction)(void (*)(void))mat, METH_FASTCALL, nullptr},
                         {"rows3", (PyCFunction)(void (*)(void))rows3, METH_FASTCALL, nullptr},
                         {"written", (PyCFunction)(void (*)(void))written, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
