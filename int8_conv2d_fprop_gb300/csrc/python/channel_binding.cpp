// channel_binding.cpp -- argument marshalling of the channel operators: torch
// tensors to the matrix descriptors of the C ABI, outputs and workspaces from
// torch's allocator, and the calls.  (In C++ because the smallest operators
// take a few microseconds: reading the tensors' attributes from Python costs
// more than the kernels.)
//
// Every function takes positional arguments only, returns its result or the
// conv_status (an int) of a refused call, and raises ValueError for tensors
// that no descriptor can say.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "int8conv.h"

namespace {

int32_t type_code(at::ScalarType t) {
    switch (t) {
        case at::kChar: return CONV_INT8;
        case at::kInt: return CONV_INT32;
        case at::kFloat: return CONV_FLOAT32;
        case at::kHalf: return CONV_FLOAT16;
        case at::kBFloat16: return CONV_BFLOAT16;
        default: return 0;  // refused by the library
    }
}

bool fail(const char *what, const char *why) {
    PyErr_Format(PyExc_ValueError, "%s %s", what, why);
    return false;
}

// What the tensors of one call have in common.
struct Common {
    const at::Tensor *first = nullptr;

    // Kernels run on one device and take addresses on trust, and the values
    // as they stand there; autograd does not see these calls.
    bool admit(const at::Tensor &t, const char *what) {
        if (!first) first = &t;
        if (t.is_neg() || t._is_zerotensor())
            return fail(what, "is a lazy view whose memory does not hold its values; clone it");
        if (t.requires_grad() && at::GradMode::is_enabled())
            return fail(what, "requires a gradient, which this call would not record: detach it, or call under "
                              "torch.no_grad() and make the gradients with the *_grad calls");
        return t.device() == first->device() || fail(what, "must be on the device of the call's other tensors");
    }
};

// The tensor behind a Python argument; NULL (no error set) for None.
const at::Tensor *tensor(Common &all, PyObject *o, const char *what, bool *ok) {
    *ok = true;
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch tensor", what);
        *ok = false;
        return nullptr;
    }
    const at::Tensor *t = &THPVariable_Unpack(o);
    *ok = t->is_cuda() ? all.admit(*t, what) : fail(what, "must be a CUDA tensor");
    return t;
}

// A tensor [..., C] as the matrix of its leading dims by C.
struct Matrix {
    conv_matrix_desc d{};
    void *p = nullptr;
    const at::Tensor *t = nullptr;
    const conv_matrix_desc *desc() const { return t ? &d : nullptr; }

    bool read(Common &all, PyObject *o, const char *what, bool required) {
        bool ok;
        t = tensor(all, o, what, &ok);
        if (!ok) return false;
        if (!t) return !required || fail(what, "is required");
        return read(*t, what);
    }

    bool read(const at::Tensor &u, const char *what) {
        t = &u;
        const auto sizes = u.sizes(), strides = u.strides();
        const int64_t dims = (int64_t)sizes.size();
        if (dims == 0) return fail(what, "must have at least one dimension");
        int64_t rows = 1, row_stride = 0;
        const bool empty = u.numel() == 0;
        for (int64_t i = dims - 2; i >= 0; --i) {
            if (sizes[i] != 1) {
                if (rows == 1) row_stride = strides[i];
                else if (!empty && strides[i] != row_stride * rows)
                    return fail(what, "has leading dimensions without a common stride; make it contiguous");
            }
            rows *= sizes[i];
        }
        d.dtype = type_code(u.scalar_type());
        d.reserved = 0;
        d.rows = rows;
        d.cols = sizes[dims - 1];
        d.row_stride = row_stride;
        d.col_stride = strides[dims - 1];
        // (a tensor always lies inside its storage: the capacity is its own extent)
        const int64_t last = empty ? 0 : (rows - 1) * d.row_stride + (d.cols - 1) * d.col_stride + 1;
        d.capacity_bytes = last > 0 ? (uint64_t)last * u.element_size() : 0;
        p = u.data_ptr();
        return true;
    }
};

// A contiguous vector of n elements, or none.
struct Vector {
    void *p = nullptr;
    int32_t type = 0;
    const at::Tensor *t = nullptr;
    bool read(Common &all, PyObject *o, const char *what, int64_t n) {
        bool ok;
        t = tensor(all, o, what, &ok);
        if (!ok) return false;
        if (!t) return true;
        if (t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1)) {
            PyErr_Format(PyExc_ValueError, "%s must be a contiguous CUDA vector of %lld elements", what, (long long)n);
            return false;
        }
        p = t->data_ptr();
        type = type_code(t->scalar_type());
        return true;
    }
    bool read_float(Common &all, PyObject *o, const char *what, int64_t n) {
        if (!read(all, o, what, n)) return false;
        return !p || type == CONV_FLOAT32 || fail(what, "must be float32");
    }
};

// Whether the parameter vectors that are there hold floats.  The library is
// told one type for them and takes their addresses on trust: a vector of a type
// without a code has to be refused here.
bool float_types(std::initializer_list<const Vector *> all) {
    for (const Vector *v : all)
        if (v->p && v->type != CONV_FLOAT32 && v->type != CONV_FLOAT16 && v->type != CONV_BFLOAT16) return false;
    return true;
}

// An activation code; -1 for a number that is none (its lower 32 bits
// may be one).
bool activation_code(PyObject *o, int32_t *code) {
    int overflow = 0;
    const long v = PyLong_AsLongAndOverflow(o, &overflow);
    if (v == -1 && PyErr_Occurred()) return false;
    *code = overflow || v < CONV_ACT_NONE || v > CONV_ACT_SILU ? -1 : (int32_t)v;
    return true;
}

// One type for the parameter vectors that are there (which hold floats).
bool one_type(std::initializer_list<const Vector *> all, int32_t *type) {
    *type = 0;
    for (const Vector *v : all) {
        if (!v->p) continue;
        if (*type && *type != v->type) {
            PyErr_SetString(PyExc_ValueError, "gain, shift and their gradients must have one type");
            return false;
        }
        *type = v->type;
    }
    if (!*type) *type = CONV_FLOAT32;
    return true;
}

// The device and stream of a call: `stream` is an address or None (the
// current stream).  Memory for a call on a given stream is allocated on that
// stream, so that the allocator hands it out again only behind the call.
struct Call {
    c10::cuda::CUDAGuard device;
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    cudaStream_t stream;
    c10::Device where;

    Call(const at::Tensor &x, PyObject *given)
        : device(x.device()), stream(nullptr), where(x.device()) {
        if (given == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(where.index()).stream();
        } else {
            stream = (cudaStream_t)PyLong_AsVoidPtr(given);
            guard.emplace(c10::cuda::getStreamFromExternal(stream, where.index()));
        }
    }
    at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type) const {
        return at::empty(sizes, at::TensorOptions().dtype(type).device(where));
    }
};

// The caller's workspace where it is large enough, else one of the call's.
struct Workspace {
    at::Tensor own;
    void *p = nullptr;
    size_t bytes = 0;
    // (before there is a call, so that nothing has touched the device yet)
    static bool admit(Common &all, PyObject *given) {
        if (!THPVariable_Check(given)) return true;
        const at::Tensor &t = THPVariable_Unpack(given);
        return !t.is_cuda() || all.admit(t, "workspace");
    }
    bool take(Common &all, const Call &c, PyObject *given, size_t need) {
        if (need == 0) return true;
        bool ok;
        const at::Tensor *t = tensor(all, given, "workspace", &ok);
        if (!ok) return false;
        if (t && t->is_contiguous() && (size_t)t->nbytes() >= need) {
            p = t->data_ptr();
            bytes = t->nbytes();
            return true;
        }
        own = c.empty({(int64_t)need}, at::kByte);
        p = own.data_ptr();
        bytes = need;
        return true;
    }
};

bool count(Py_ssize_t have, Py_ssize_t want) {
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "takes %zd arguments, got %zd", want, have);
    return false;
}

// Tells autograd that a tensor's values changed, as an in-place operation
// does: graphs that saved them refuse to go back.
void changed(std::initializer_list<const at::Tensor *> outputs) {
    for (const at::Tensor *t : outputs)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

PyObject *status(conv_status st) { return PyLong_FromLong(st); }

// linear(x, w, bias, activation, residual, preact, out, workspace, stream) -> out
PyObject *linear(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 9)) return nullptr;
    Common all;
    Matrix x, w, r, z, y;
    Vector b;
    if (!x.read(all, arg[0], "x", true) || !w.read(all, arg[1], "w", true) || !b.read(all, arg[2], "bias", w.d.rows) ||
        !r.read(all, arg[4], "residual", false) || !z.read(all, arg[5], "preact", false) || !y.read(all, arg[6], "out", false) ||
        !Workspace::admit(all, arg[7]))
        return nullptr;
    conv_linear_params p{};
    if (!activation_code(arg[3], &p.activation)) return nullptr;
    if (p.activation < 0) return status(CONV_ERR_BAD_PARAM);
    p.bias_dtype = b.type;
    const Call c(*x.t, arg[8]);
    at::Tensor made;
    if (!y.t) {
        at::DimVector sizes(x.t->sizes().begin(), x.t->sizes().end());
        sizes.back() = w.d.rows;
        made = c.empty(sizes, x.t->scalar_type());
        if (!y.read(made, "out")) return nullptr;
    }
    size_t need = 0;
    conv_status st = conv_linear_workspace_size(&x.d, x.p, &w.d, w.p, &need);
    if (st) return status(st);
    Workspace ws;
    if (!ws.take(all, c, arg[7], need)) return nullptr;
    st = conv_linear(&x.d, x.p, &w.d, w.p, b.p, r.desc(), r.p, z.desc(), z.p, &y.d, y.p, &p, ws.p, ws.bytes, c.stream);
    if (st) return status(st);
    if (made.defined()) y.t = nullptr;
    changed({z.t, y.t});
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(arg[6]);
    return arg[6];
    END_HANDLE_TH_ERRORS
}

// linear_grad(dy, x, w, preact, activation, dx, dw, dbias, workspace, stream) -> None
PyObject *linear_grad(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 10)) return nullptr;
    Common all;
    Matrix dy, x, w, z, dx, dw;
    Vector db;
    if (!dy.read(all, arg[0], "dy", true) || !x.read(all, arg[1], "x", true) || !w.read(all, arg[2], "w", true) ||
        !z.read(all, arg[3], "preact", false) || !dx.read(all, arg[5], "dx", false) || !dw.read(all, arg[6], "dw", false) ||
        !db.read(all, arg[7], "dbias", w.d.rows) || !Workspace::admit(all, arg[8]))
        return nullptr;
    conv_linear_params p{};
    if (!activation_code(arg[4], &p.activation)) return nullptr;
    if (p.activation < 0) return status(CONV_ERR_BAD_PARAM);
    p.bias_dtype = db.type;
    const Call c(*x.t, arg[9]);
    size_t need = 0;
    conv_status st = conv_linear_grad_workspace_size(&dy.d, dy.p, &x.d, x.p, &w.d, w.p, &p, &need);
    if (st) return status(st);
    Workspace ws;
    if (!ws.take(all, c, arg[8], need)) return nullptr;
    st = conv_linear_grad(&dy.d, dy.p, &x.d, x.p, &w.d, w.p, z.desc(), z.p, dx.desc(), dx.p, dw.desc(), dw.p, db.p, &p,
                          ws.p, ws.bytes, c.stream);
    if (st) return status(st);
    changed({dx.t, dw.t, db.t});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// layer_norm(x, gain, shift, eps, scale, out, mean, rstd, stream) -> out
PyObject *layer_norm(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 9)) return nullptr;
    Common all;
    Matrix x, y;
    Vector g, h, mean, rstd;
    if (!x.read(all, arg[0], "x", true) || !g.read(all, arg[1], "gain", x.d.cols) || !h.read(all, arg[2], "shift", x.d.cols) ||
        !y.read(all, arg[5], "out", false) || !mean.read_float(all, arg[6], "mean", x.d.rows) ||
        !rstd.read_float(all, arg[7], "rstd", x.d.rows))
        return nullptr;
    conv_layer_norm_params p{};
    p.eps = (float)PyFloat_AsDouble(arg[3]);
    p.scale = (float)PyFloat_AsDouble(arg[4]);
    if (PyErr_Occurred()) return nullptr;
    if (!float_types({&g, &h})) return status(CONV_ERR_DTYPE);
    if (!one_type({&g, &h}, &p.param_dtype)) return nullptr;
    const Call c(*x.t, arg[8]);
    at::Tensor made;
    if (!y.t) {
        made = c.empty(x.t->sizes(), x.t->is_floating_point() ? x.t->scalar_type() : at::kFloat);
        if (!y.read(made, "out")) return nullptr;
    }
    const conv_status st = conv_layer_norm(&x.d, x.p, g.p, h.p, &y.d, y.p, (float *)mean.p, (float *)rstd.p, &p, c.stream);
    if (st) return status(st);
    if (made.defined()) y.t = nullptr;
    changed({y.t, mean.t, rstd.t});
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(arg[5]);
    return arg[5];
    END_HANDLE_TH_ERRORS
}

// layer_norm_grad(dy, x, gain, mean, rstd, residual_grad, dx, dgain, dshift, workspace, stream) -> None
PyObject *layer_norm_grad(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 11)) return nullptr;
    Common all;
    Matrix dy, x, r, dx;
    Vector g, mean, rstd, dg, dh;
    if (!dy.read(all, arg[0], "dy", true) || !x.read(all, arg[1], "x", true) || !g.read(all, arg[2], "gain", x.d.cols) ||
        !mean.read_float(all, arg[3], "mean", x.d.rows) || !rstd.read_float(all, arg[4], "rstd", x.d.rows) ||
        !r.read(all, arg[5], "residual_grad", false) || !dx.read(all, arg[6], "dx", false) ||
        !dg.read(all, arg[7], "dgain", x.d.cols) || !dh.read(all, arg[8], "dshift", x.d.cols) ||
        !Workspace::admit(all, arg[9]))
        return nullptr;
    conv_layer_norm_params p{};
    p.eps = 1e-5f;
    p.scale = 1.0f;
    if (!float_types({&g, &dg, &dh})) return status(CONV_ERR_DTYPE);
    if (!one_type({&g, &dg, &dh}, &p.param_dtype)) return nullptr;
    const Call c(*x.t, arg[10]);
    size_t need = 0;
    conv_status st = conv_layer_norm_grad_workspace_size(&x.d, &need);
    if (st) return status(st);
    Workspace ws;
    if (!ws.take(all, c, arg[9], need)) return nullptr;
    st = conv_layer_norm_grad(&dy.d, dy.p, &x.d, x.p, g.p, (const float *)mean.p, (const float *)rstd.p, r.desc(), r.p,
                              dx.desc(), dx.p, dg.p, dh.p, &p, ws.p, ws.bytes, c.stream);
    if (st) return status(st);
    changed({dx.t, dg.t, dh.t});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"linear", (PyCFunction)(void (*)())linear, METH_FASTCALL, nullptr},
    {"linear_grad", (PyCFunction)(void (*)())linear_grad, METH_FASTCALL, nullptr},
    {"layer_norm", (PyCFunction)(void (*)())layer_norm, METH_FASTCALL, nullptr},
    {"layer_norm_grad", (PyCFunction)(void (*)())layer_norm_grad, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_channel", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__channel(void) { return PyModule_Create(&module); }
