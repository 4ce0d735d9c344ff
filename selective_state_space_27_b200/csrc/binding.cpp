// Tensor checks of the serving operators' Python calls, compiled: a decode step
// makes a dozen of them per layer, and in Python they take longer than the kernel
// (2 requests x 80 heads: 14 us per call against 6 us on the device).
//   rows(name, t, dtype, shape, device) -> (pointer, stride of the first axis)
//   vector(name, t, n, device, dtype)   -> pointer
//   empty_like(t), scratch(bytes, t)    -> uninitialised tensors on t's device
// A None tensor has pointer and stride 0; what does not fit raises ValueError or,
// for a type, TypeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

namespace {

const char *text(PyObject *name) { return PyUnicode_Check(name) ? PyUnicode_AsUTF8(name) : "tensor"; }

bool arguments(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", want, n);
    return false;
}

bool is_tensor(PyObject *name, PyObject *t) {
    if (THPVariable_Check(t)) return true;
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %s", text(name), Py_TYPE(t)->tp_name);
    return false;
}

// What is wrong with t, in the order device, type, shape. Always null.
PyObject *refuse(PyObject *name, PyObject *t, PyObject *dtype, PyObject *shape, PyObject *device) {
    const at::Tensor &x = THPVariable_Unpack(t);
    const at::Device want = reinterpret_cast<THPDevice *>(device)->device;
    if (x.device() != want) {
        PyErr_Format(PyExc_ValueError, "%s is on %s, expected %s", text(name), x.device().str().c_str(),
                     want.str().c_str());
    } else if (x.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type) {
        PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", text(name), dtype,
                     reinterpret_cast<PyObject *>(torch::getTHPDtype(x.scalar_type())));
    } else {
        PyObject *got = PyObject_GetAttrString(t, "shape");
        if (got) {
            PyErr_Format(PyExc_ValueError, "%s must have shape %S, got %S", text(name), shape, got);
            Py_DECREF(got);
        }
    }
    return nullptr;
}

bool types(PyObject *dtype, PyObject *device) {
    if (THPDtype_Check(dtype) && THPDevice_Check(device)) return true;
    PyErr_SetString(PyExc_TypeError, "a torch.dtype and a torch.device are expected");
    return false;
}

PyObject *pair(uint64_t a, int64_t b) {
    PyObject *r = PyTuple_New(2), *p = PyLong_FromUnsignedLongLong(a), *q = PyLong_FromLongLong(b);
    if (!r || !p || !q) {
        Py_XDECREF(r);
        Py_XDECREF(p);
        Py_XDECREF(q);
        return nullptr;
    }
    PyTuple_SET_ITEM(r, 0, p);
    PyTuple_SET_ITEM(r, 1, q);
    return r;
}

uint64_t address(const at::Tensor &x) { return reinterpret_cast<uint64_t>(x.data_ptr()); }

PyObject *rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 5)) return nullptr;
    PyObject *name = a[0], *t = a[1], *dtype = a[2], *shape = a[3], *device = a[4];
    if (t == Py_None) return pair(0, 0);
    if (!is_tensor(name, t) || !types(dtype, device)) return nullptr;
    if (!PyTuple_Check(shape)) {
        PyErr_SetString(PyExc_TypeError, "the shape must be a tuple");
        return nullptr;
    }
    const at::Tensor &x = THPVariable_Unpack(t);
    const int64_t dim = x.dim();
    bool fits = x.scalar_type() == reinterpret_cast<THPDtype *>(dtype)->scalar_type &&
                x.device() == reinterpret_cast<THPDevice *>(device)->device && PyTuple_GET_SIZE(shape) == dim && dim > 0;
    for (int64_t i = 0; fits && i < dim; ++i) {
        const long long size = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (size == -1 && PyErr_Occurred()) PyErr_Clear();   // (a name in place of a size: it fits nothing)
        fits = x.size(i) == size;
    }
    if (!fits) return refuse(name, t, dtype, shape, device);
    int64_t inner = 1;
    for (int64_t i = dim - 1; i > 0; --i) {
        if (x.size(i) > 1 && x.stride(i) != inner && x.numel() > 0) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous behind its first axis", text(name));
            return nullptr;
        }
        inner *= x.size(i);
    }
    return pair(address(x), x.size(0) <= 1 || x.numel() == 0 ? inner : x.stride(0));
    END_HANDLE_TH_ERRORS
}

PyObject *vector(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 5)) return nullptr;
    PyObject *name = a[0], *t = a[1], *device = a[3], *dtype = a[4];
    if (t == Py_None) return PyLong_FromLong(0);
    if (!is_tensor(name, t) || !types(dtype, device)) return nullptr;
    const long long count = PyLong_AsLongLong(a[2]);
    if (count == -1 && PyErr_Occurred()) return nullptr;
    const at::Tensor &x = THPVariable_Unpack(t);
    if (x.scalar_type() != reinterpret_cast<THPDtype *>(dtype)->scalar_type ||
        x.device() != reinterpret_cast<THPDevice *>(device)->device || x.dim() != 1 || x.size(0) != count) {
        PyObject *shape = PyTuple_Pack(1, a[2]);
        if (shape) {
            refuse(name, t, dtype, shape, device);
            Py_DECREF(shape);
        }
        return nullptr;
    }
    if (!x.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", text(name));
        return nullptr;
    }
    return PyLong_FromUnsignedLongLong(address(x));
    END_HANDLE_TH_ERRORS
}

PyObject *empty_like(PyObject *, PyObject *t) {
    HANDLE_TH_ERRORS
    if (!is_tensor(Py_None, t)) return nullptr;
    const at::Tensor &x = THPVariable_Unpack(t);
    return THPVariable_Wrap(at::empty(x.sizes(), x.options()));
    END_HANDLE_TH_ERRORS
}

PyObject *scratch(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 2) || !is_tensor(Py_None, a[1])) return nullptr;
    const long long bytes = PyLong_AsLongLong(a[0]);
    if (bytes == -1 && PyErr_Occurred()) return nullptr;
    return THPVariable_Wrap(at::empty({bytes}, THPVariable_Unpack(a[1]).options().dtype(at::kByte)));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rows)), METH_FASTCALL,
     "rows(name, t, dtype, shape, device): (pointer, stride of the first axis)."},
    {"vector", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(vector)), METH_FASTCALL,
     "vector(name, t, n, device, dtype): pointer."},
    {"empty_like", empty_like, METH_O, "An uninitialised contiguous tensor of t's sizes, type and device."},
    {"scratch", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(scratch)), METH_FASTCALL,
     "scratch(bytes, t): uninitialised bytes on t's device."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Tensor checks of the serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
