// Checks of tensor arguments for the Python operators (ops.py), and the versions of the tensors that they write, as a CPython
// extension: type, size, device and layout of a tensor are read from the tensor itself instead of attribute by attribute through Python (some 0.4 us a tensor; a call
// takes up to twelve, and a small call is as long as its host side).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/GradMode.h>
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

// A tuple of the addresses of contiguous tensors of n elements each, from `each` arguments a tensor: its name, itself, its type
// (int32 where each is three) and n.
PyObject* addresses(PyObject* const* a, Py_ssize_t na, int each) {
    if (na < 1 || na % each != 1) return PyErr_Format(PyExc_TypeError, "a device, and %d arguments for each tensor", each);
    return guarded([&]() -> PyObject* {
        const long dev = PyLong_AsLong(a[0]);
        if (PyErr_Occurred()) return nullptr;
        PyObject* out = PyTuple_New(na / each);
        if (!out) return nullptr;
        for (Py_ssize_t i = 0; i < na / each; ++i) {
            PyObject* const* e = a + 1 + each * i;
            const at::Tensor* t = tensor(e[1]);
            const long long n = PyLong_AsLongLong(e[each - 1]);
            if (!t || PyErr_Occurred()) {
                Py_DECREF(out);
                return nullptr;
            }
            if (!(each == 3 ? t->scalar_type() == at::kInt : of_type(*t, e[2])) || t->numel() != n || t->get_device() != dev ||
                !t->is_contiguous()) {
                Py_DECREF(out);
                return refuse(e[0], each == 3 ? PyUnicode_FromFormat("a contiguous torch.int32 tensor of %lld elements", n)
                                              : PyUnicode_FromFormat("a contiguous %S tensor of %lld elements", e[2], n),
                              dev, e[1]);
            }
            PyObject* address = PyLong_FromVoidPtr(t->data_ptr());
            if (!address) {
                Py_DECREF(out);
                return nullptr;
            }
            PyTuple_SET_ITEM(out, i, address);
        }
        return out;
    });
}
// ints(dev, name, t, n, ...), flats(dev, name, t, dtype, n, ...)
PyObject* ints(PyObject*, PyObject* const* a, Py_ssize_t na) { return addresses(a, na, 3); }
PyObject* flats(PyObject*, PyObject* const* a, Py_ssize_t na) { return addresses(a, na, 4); }

// free_of_grad(t, ...): whether none of the tensors (or None) would record a gradient
PyObject* free_of_grad(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded([&]() -> PyObject* {
        if (c10::GradMode::is_enabled())
            for (Py_ssize_t i = 0; i < na; ++i) {
                if (a[i] == Py_None) continue;
                const at::Tensor* t = tensor(a[i]);
                if (!t) return nullptr;
                if (t->requires_grad()) Py_RETURN_FALSE;
            }
        Py_RETURN_TRUE;
    });
}

// caches(k, v, dev): (dtype code, layers, pages, heads, hd, elements between layers) of two caches of pages of 64 tokens
PyObject* caches(PyObject*, PyObject* const* a, Py_ssize_t na) {
    if (!args(na, 3)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor *k = tensor(a[0]), *v = k ? tensor(a[1]) : nullptr;
        const long dev = PyLong_AsLong(a[2]);
        if (!v || PyErr_Occurred()) return nullptr;
        auto bad = [](const char* m) -> PyObject* {
            PyErr_SetString(PyExc_ValueError, m);
            return nullptr;
        };
        const bool bf16 = k->scalar_type() == at::kBFloat16;
        if (!bf16 && k->scalar_type() != at::kFloat) return bad("k_cache must be float32 or bfloat16");
        const int64_t d = k->dim();
        if (v->scalar_type() != k->scalar_type() || v->sizes() != k->sizes() || (d != 4 && d != 5) || k->size(d - 2) != 64)
            return bad("k_cache and v_cache must be alike, [pages, H_kv, 64, hd] or [layers, pages, H_kv, 64, hd]");
        if (k->get_device() != dev || v->get_device() != dev) return bad("k_cache and v_cache must be on the other tensors' device");
        const int64_t pages = k->size(d - 4), heads = k->size(d - 3), hd = k->size(d - 1), layer = pages * heads * 64 * hd;
        for (const at::Tensor* t : {k, v}) {  // a layer is contiguous
            int64_t want = 1;
            for (int64_t i = d - 1; i >= d - 4; --i) {
                if (t->size(i) != 1 && t->stride(i) != want) return bad("a layer of k_cache and v_cache must be contiguous");
                want *= t->size(i);
            }
        }
        const int64_t layers = d == 5 ? k->size(0) : 1;
        if (layers < 1) return bad("k_cache and v_cache must hold a layer");
        if (layers > 1 && k->stride(0) != v->stride(0)) return bad("k_cache and v_cache must have one stride between layers");
        return Py_BuildValue("iLLLLL", bf16 ? 1 : 0, (long long)layers, (long long)pages, (long long)heads, (long long)hd,
                             layers > 1 ? (long long)k->stride(0) : (long long)layer);
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
                         {"ints", (PyCFunction)(void (*)(void))ints, METH_FASTCALL, nullptr},
                         {"flats", (PyCFunction)(void (*)(void))flats, METH_FASTCALL, nullptr},
                         {"free_of_grad", (PyCFunction)(void (*)(void))free_of_grad, METH_FASTCALL, nullptr},
                         {"caches", (PyCFunction)(void (*)(void))caches, METH_FASTCALL, nullptr},
                         {"written", (PyCFunction)(void (*)(void))written, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
