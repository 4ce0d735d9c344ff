// Tensor checks of the serving operators' Python calls, compiled: a decode step
// makes a dozen of them per layer, and in Python they take longer than the kernel
// (2 requests x 80 heads: 14 us per call against 6 us on the device). The norms,
// the calls with the least work per tensor, are marshalled here altogether.
//   rows(name, t, dtype, shape, device) -> (pointer, stride of the first axis)
//   vector(name, t, n, device, dtype)   -> pointer
//   empty_like(t)                       -> an uninitialised tensor like it
//   norm_fwd(entry point, stream, arguments of serving.norm_fwd) -> (status, y, residual_out)
//   norm_bwd(entry point, its workspace query, stream, arguments) -> (status, dx, dz, dresidual, dweight)
//   ssd_packed(entry point, its workspace query, stream, packed arguments, x, workspace, replace) -> (status, workspace used)
// A None tensor has pointer and stride 0; what does not fit raises ValueError or,
// for a type, TypeError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstring>
#include <string>

#include <ATen/ATen.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mambascan.h"

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

// What can be wrong with a call of the norms; the message is raised as its type says.
struct Refused {
    PyObject *type;
    std::string text;
};

const at::Tensor *optional(const char *name, PyObject *t) {
    if (t == Py_None) return nullptr;
    if (!THPVariable_Check(t)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
    return &THPVariable_Unpack(t);
}

std::string sizes(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

// (rows, dim) of `type` on x's device, channels contiguous.
template <typename P>
void matrix(const char *name, const at::Tensor &t, at::ScalarType type, const at::Tensor &x, P &ptr, int64_t &stride) {
    if (t.device() != x.device())
        throw Refused{PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected " + x.device().str()};
    if (t.scalar_type() != type)
        throw Refused{PyExc_TypeError, std::string(name) + " must be " + at::toString(type) + ", got " +
                                           at::toString(t.scalar_type())};
    if (t.sizes() != x.sizes())
        throw Refused{PyExc_ValueError, std::string(name) + " must have shape " + sizes(x.sizes()) + ", got " +
                                            sizes(t.sizes())};
    if (t.size(1) > 1 && t.stride(1) != 1 && t.numel() > 0)
        throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous behind its first axis"};
    ptr = static_cast<P>(t.data_ptr());
    stride = t.size(0) <= 1 || t.numel() == 0 ? t.size(1) : t.stride(0);
}

int32_t code(const char *name, const at::Tensor &t) {
    if (t.scalar_type() == at::kFloat) return MS_F32;
    if (t.scalar_type() == at::kBFloat16) return MS_BF16;
    throw Refused{PyExc_TypeError, std::string(name) + ": unsupported dtype " + at::toString(t.scalar_type()) +
                                       " (float32 or bfloat16)"};
}

// The arguments that forward and backward share.
const at::Tensor &norm_arguments(ms_norm_args &a, PyObject *xo, PyObject *weight, PyObject *zo, PyObject *scale,
                                 PyObject *eps, PyObject *group, PyObject *gate_first) {
    const at::Tensor *x = optional("x", xo);
    if (!x || !x->is_cuda()) throw Refused{PyExc_ValueError, "x must be a CUDA tensor"};
    if (x->dim() != 2) throw Refused{PyExc_ValueError, "x must have 2 dimensions"};
    a.in_dtype = a.residual_dtype = code("x", *x);
    a.rows = x->size(0);
    a.dim = x->size(1);
    a.group_size = group == Py_None ? a.dim : PyLong_AsLongLong(group);
    a.eps = static_cast<float>(PyFloat_AsDouble(eps));
    a.residual_scale = static_cast<float>(PyFloat_AsDouble(scale));
    a.gate_first = PyObject_IsTrue(gate_first);
    if (PyErr_Occurred()) throw Refused{nullptr, ""};
    matrix("x", *x, x->scalar_type(), *x, a.x, a.x_row_stride);
    if (const at::Tensor *z = optional("z", zo)) matrix("z", *z, x->scalar_type(), *x, a.z, a.z_row_stride);
    if (const at::Tensor *w = optional("weight", weight)) {
        if (w->device() != x->device())
            throw Refused{PyExc_ValueError, "weight is on " + w->device().str() + ", expected " + x->device().str()};
        if (w->scalar_type() != at::kFloat) throw Refused{PyExc_TypeError, "weight must be torch.float32"};
        if (w->dim() != 1 || w->size(0) != a.dim || !w->is_contiguous())
            throw Refused{PyExc_ValueError, "weight must be contiguous with shape (" + std::to_string(a.dim) + ",)"};
        a.weight = static_cast<const float *>(w->data_ptr());
    }
    return *x;
}

int32_t residual_code(const at::Tensor &r, const at::Tensor &x) {
    if (r.scalar_type() != x.scalar_type() && r.scalar_type() != at::kFloat)
        throw Refused{PyExc_TypeError, std::string("the residual must have x's dtype or torch.float32, got ") +
                                           at::toString(r.scalar_type())};
    return code("residual", r);
}

PyObject *raise(const Refused &r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
    return nullptr;
}

template <typename F>
F entry(PyObject *address) {
    return reinterpret_cast<F>(PyLong_AsVoidPtr(address));
}

PyObject *norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 12)) return nullptr;
    try {
        const auto fn = entry<ms_status (*)(const ms_norm_args *, void *)>(a[0]);
        void *stream = PyLong_AsVoidPtr(a[1]);
        ms_norm_args p{};
        const at::Tensor &x = norm_arguments(p, a[2], a[3], a[4], a[6], a[7], a[8], a[9]);
        const at::Tensor *res = optional("residual", a[5]), *out = optional("out", a[10]),
                         *total = optional("residual_out", a[11]);
        if (!res && total) throw Refused{PyExc_ValueError, "residual_out needs a residual"};
        at::Tensor y = out ? *out : at::empty(x.sizes(), x.options()), ro;
        matrix("out", y, x.scalar_type(), x, p.y, p.y_row_stride);
        if (res) {
            p.residual_dtype = residual_code(*res, x);
            matrix("residual", *res, res->scalar_type(), x, p.residual, p.residual_row_stride);
            ro = total ? *total : at::empty(x.sizes(), res->options());
            matrix("residual_out", ro, res->scalar_type(), x, p.residual_out, p.residual_out_row_stride);
        }
        if (PyErr_Occurred()) return nullptr;
        ms_status status;
        Py_BEGIN_ALLOW_THREADS
        status = fn(&p, stream);
        Py_END_ALLOW_THREADS
        PyObject *r = PyTuple_New(3);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(y));
        PyTuple_SET_ITEM(r, 2, res ? THPVariable_Wrap(ro) : Py_NewRef(Py_None));
        return r;
    } catch (const Refused &r) {
        return raise(r);
    }
    END_HANDLE_TH_ERRORS
}

PyObject *norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 14)) return nullptr;
    try {
        const auto fn = entry<ms_status (*)(const ms_norm_args *, const ms_norm_bwd_args *, void *, size_t, void *)>(a[0]);
        const auto query = entry<ms_status (*)(const ms_norm_args *, size_t *)>(a[1]);
        void *stream = PyLong_AsVoidPtr(a[2]);
        ms_norm_args p{};
        ms_norm_bwd_args g{};
        const at::Tensor &x = norm_arguments(p, a[4], a[5], a[6], a[9], a[10], a[11], a[12]);
        const at::Tensor *dy = optional("dy", a[3]), *ro = optional("residual_out", a[7]),
                         *dro = optional("dresidual_out", a[8]), *given = optional("workspace", a[13]);
        if (!dy) throw Refused{PyExc_ValueError, "dy is needed"};
        if (!ro && dro) throw Refused{PyExc_ValueError, "dresidual_out needs residual_out"};
        matrix("dy", *dy, x.scalar_type(), x, g.dy, g.dy_row_stride);
        at::Tensor dx = at::empty(x.sizes(), x.options()), dz, dres, dw, scratch;
        matrix("dx", dx, x.scalar_type(), x, g.dx, g.dx_row_stride);
        if (ro) {
            p.residual_dtype = residual_code(*ro, x);
            matrix("residual_out", *ro, ro->scalar_type(), x, p.residual_out, p.residual_out_row_stride);
            if (dro) matrix("dresidual_out", *dro, ro->scalar_type(), x, g.dresidual_out, g.dresidual_out_row_stride);
            dres = at::empty(x.sizes(), ro->options());
            matrix("dresidual", dres, ro->scalar_type(), x, g.dresidual, g.dresidual_row_stride);
        }
        if (p.z) {
            dz = at::empty(x.sizes(), x.options());
            matrix("dz", dz, x.scalar_type(), x, g.dz, g.dz_row_stride);
        }
        ms_status status = MS_OK;
        void *space = nullptr;
        size_t bytes = 0;
        if (p.weight) {
            dw = at::empty({p.dim}, x.options().dtype(at::kFloat));
            g.dweight = static_cast<float *>(dw.data_ptr());
            if (given && (given->scalar_type() != at::kByte || given->device() != x.device() || !given->is_contiguous()))
                throw Refused{PyExc_ValueError, "workspace must be a contiguous uint8 tensor on " + x.device().str()};
            status = query(&p, &bytes);
            if (status == MS_OK && bytes) {
                if (given && static_cast<size_t>(given->numel()) >= bytes) {
                    space = given->data_ptr();
                } else {
                    scratch = at::empty({static_cast<int64_t>(bytes)}, x.options().dtype(at::kByte));
                    space = scratch.data_ptr();
                }
            }
        }
        if (PyErr_Occurred()) return nullptr;
        if (status == MS_OK) {
            Py_BEGIN_ALLOW_THREADS
            status = fn(&p, &g, space, bytes, stream);
            Py_END_ALLOW_THREADS
        }
        PyObject *r = PyTuple_New(5);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
        const at::Tensor *results[] = {&dx, &dz, &dres, &dw};
        for (int i = 0; i < 4; ++i)
            PyTuple_SET_ITEM(r, i + 1, results[i]->defined() ? THPVariable_Wrap(*results[i]) : Py_NewRef(Py_None));
        return r;
    } catch (const Refused &r) {
        return raise(r);
    }
    END_HANDLE_TH_ERRORS
}

// The workspace's size, a workspace of that size where none is given or (replace) the given
// one is too small, and the call. Without replace the call refuses one that is too small.
PyObject *ssd_packed(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!arguments(n, 7)) return nullptr;
    try {
        const auto fn = entry<ms_status (*)(const ms_ssd_packed_args *, void *, size_t, void *)>(a[0]);
        const auto query = entry<ms_status (*)(const ms_ssd_packed_args *, size_t *)>(a[1]);
        void *stream = PyLong_AsVoidPtr(a[2]);
        char *bytes = nullptr;
        Py_ssize_t length = 0;
        const int replace = PyObject_IsTrue(a[6]);
        if (replace < 0 || PyBytes_AsStringAndSize(a[3], &bytes, &length) < 0 || PyErr_Occurred()) return nullptr;
        const at::Tensor *x = optional("x", a[4]), *given = optional("workspace", a[5]);
        if (!x || length != sizeof(ms_ssd_packed_args)) throw Refused{PyExc_ValueError, "the packed arguments do not fit"};
        ms_ssd_packed_args p;
        std::memcpy(&p, bytes, sizeof(p));
        if (given && (given->scalar_type() != at::kByte || given->device() != x->device() || !given->is_contiguous()))
            throw Refused{PyExc_ValueError, "workspace must be a contiguous uint8 tensor on " + x->device().str()};
        size_t need = 0;
        ms_status status = query(&p, &need);
        at::Tensor space;
        if (status == MS_OK) {
            space = given && (!replace || static_cast<size_t>(given->numel()) >= need)
                        ? *given
                        : at::empty({static_cast<int64_t>(need)}, x->options().dtype(at::kByte));
            void *at = space.data_ptr();
            const size_t size = static_cast<size_t>(space.numel());
            Py_BEGIN_ALLOW_THREADS
            status = fn(&p, at, size, stream);
            Py_END_ALLOW_THREADS
        }
        PyObject *r = PyTuple_New(2);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, PyLong_FromLong(status));
        PyTuple_SET_ITEM(r, 1, space.defined() ? THPVariable_Wrap(space) : Py_NewRef(Py_None));
        return r;
    } catch (const Refused &r) {
        return raise(r);
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(rows)), METH_FASTCALL,
     "rows(name, t, dtype, shape, device): (pointer, stride of the first axis)."},
    {"vector", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(vector)), METH_FASTCALL,
     "vector(name, t, n, device, dtype): pointer."},
    {"empty_like", empty_like, METH_O, "An uninitialised contiguous tensor of t's sizes, type and device."},
    {"norm_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_fwd)), METH_FASTCALL,
     "norm_fwd(entry point, stream, x, weight, z, residual, scale, eps, group_size, gate_first, out, residual_out)."},
    {"norm_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_bwd)), METH_FASTCALL,
     "norm_bwd(entry point, query, stream, dy, x, weight, z, residual_out, dresidual_out, scale, eps, group_size, "
     "gate_first, workspace)."},
    {"ssd_packed", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(ssd_packed)), METH_FASTCALL,
     "ssd_packed(entry point, query, stream, packed arguments, x, workspace, replace)."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Tensor checks of the serving operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
