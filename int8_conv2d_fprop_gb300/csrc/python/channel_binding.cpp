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
#include <ATen/ops/empty_strided.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>
#include <vector>

#include "int8conv.h"

namespace {

int32_t type_code(at::ScalarType t) {
    switch (t) {
        case at::kChar: return CONV_INT8;
        case at::kInt: return CONV_INT32;
        case at::kFloat: return CONV_FLOAT32;
        case at::kHalf: return CONV_FLOAT16;
        case at::kBFloat16: return CONV_BFLOAT16;
        case at::kFloat8_e4m3fn: return CONV_FLOAT8_E4M3;
        case at::kFloat8_e5m2: return CONV_FLOAT8_E5M2;
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

// The tensor type of a code that an entry point allocates an output in.
bool scalar_type(PyObject *o, at::ScalarType *type) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    switch (v) {
        case CONV_FLOAT32: *type = at::kFloat; return true;
        case CONV_FLOAT16: *type = at::kHalf; return true;
        case CONV_BFLOAT16: *type = at::kBFloat16; return true;
        case CONV_FLOAT8_E4M3: *type = at::kFloat8_e4m3fn; return true;
        case CONV_FLOAT8_E5M2: *type = at::kFloat8_e5m2; return true;
        default: PyErr_SetString(PyExc_ValueError, "dtype is not one this call makes"); return false;
    }
}

// A Python number as a 32-bit float; one that would become an infinity there
// would mean something else.
bool number(PyObject *o, float *v) {
    const double d = PyFloat_AsDouble(o);
    *v = (float)d;
    if (PyErr_Occurred()) return false;
    if (std::isinf(*v) && !std::isinf(d)) {
        PyErr_SetString(PyExc_ValueError, "a number is beyond the range of 32-bit floats");
        return false;
    }
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
    // A matrix [..., cols] of like's leading dims (or of `rows` alone), rows and columns these strides apart.
    at::Tensor matrix(const at::Tensor *like, int64_t rows, int64_t cols, int64_t row_stride, int64_t col_stride,
                      at::ScalarType type) const {
        at::DimVector sizes, strides;
        if (like) {
            sizes.assign(like->sizes().begin(), like->sizes().end());
            strides.resize(sizes.size());
            int64_t step = row_stride;
            for (int64_t i = (int64_t)sizes.size() - 2; i >= 0; --i) {
                strides[i] = step;
                step *= sizes[i];
            }
            sizes.back() = cols;
            strides.back() = col_stride;
        } else {
            sizes = {rows, cols};
            strides = {row_stride, col_stride};
        }
        return at::empty_strided(sizes, strides, at::TensorOptions().dtype(type).device(where));
    }
};

int64_t blocks_of(int64_t n, int64_t of) { return (n + of - 1) / of; }

// The scales of [rows, cols] in blocks of `tile` rows: neighbouring rows' next to one another.
at::Tensor scales_for(const Call &c, const at::Tensor *like, int64_t rows, int64_t cols, int64_t tile) {
    const int64_t lines = blocks_of(rows, tile);
    return c.matrix(tile == 1 ? like : nullptr, lines, blocks_of(cols, 128), 1, std::max<int64_t>(lines, 1), at::kFloat);
}
// 8-bit values in rows of a multiple of 16 bytes, as the products read them in place.
at::Tensor eight_bit_for(const Call &c, const at::Tensor *like, int64_t rows, int64_t cols, at::ScalarType type) {
    return c.matrix(like, rows, cols, std::max<int64_t>(blocks_of(cols, 16), 1) * 16, 1, type);
}

// A result that was allocated here, or the caller's own (borrowed from its argument).
PyObject *result(at::Tensor &made, PyObject *given) {
    if (made.defined()) return THPVariable_Wrap(std::move(made));
    Py_INCREF(given);
    return given;
}

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

// quantize(x, preact, activation, tile, dtype, rows, columns, out, scale, out_t, scale_t, stream)
//     -> (out, scale) of rows, of columns, or of both
PyObject *quantize(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 12)) return nullptr;
    Common all;
    Matrix x, z, m[4];  // q, scale, qt, scale_t
    static const char *const names[] = {"out", "scale", "out_t", "scale_t"};
    if (!x.read(all, arg[0], "x", true) || !z.read(all, arg[1], "preact", false)) return nullptr;
    for (int i = 0; i < 4; ++i)
        if (!m[i].read(all, arg[7 + i], names[i], false)) return nullptr;
    conv_quantize_params p{};
    if (!activation_code(arg[2], &p.activation)) return nullptr;
    if (p.activation < 0) return status(CONV_ERR_BAD_PARAM);
    const long tile = PyLong_AsLong(arg[3]);
    if (tile == -1 && PyErr_Occurred()) return nullptr;
    if (tile != 1 && tile != 128) return status(CONV_ERR_BAD_PARAM);
    p.tile = (int32_t)tile;
    at::ScalarType type;
    if (!scalar_type(arg[4], &type)) return nullptr;
    const bool want[2] = {PyObject_IsTrue(arg[5]) == 1, PyObject_IsTrue(arg[6]) == 1};
    const int64_t rows = x.d.rows, cols = x.d.cols;
    const Call c(*x.t, arg[11]);
    at::Tensor made[4];
    for (int f = 0; f < 2; ++f) {
        if (!want[f]) {
            if (m[2 * f].t || m[2 * f + 1].t) {
                PyErr_Format(PyExc_ValueError, "%s is given, but not wanted", names[m[2 * f].t ? 2 * f : 2 * f + 1]);
                return nullptr;
            }
            continue;
        }
        const int64_t a = f ? cols : rows, b = f ? rows : cols;
        const at::Tensor *like = f ? nullptr : x.t;
        if (!m[2 * f].t) {
            made[2 * f] = eight_bit_for(c, like, a, b, type);
            if (!m[2 * f].read(made[2 * f], names[2 * f])) return nullptr;
        }
        if (!m[2 * f + 1].t) {
            made[2 * f + 1] = scales_for(c, like, a, b, tile);
            if (!m[2 * f + 1].read(made[2 * f + 1], names[2 * f + 1])) return nullptr;
        }
    }
    const conv_status st = conv_quantize(&x.d, x.p, z.desc(), z.p, m[0].desc(), m[0].p, m[1].desc(), m[1].p, m[2].desc(),
                                         m[2].p, m[3].desc(), m[3].p, &p, c.stream);
    if (st) return status(st);
    PyObject *r = PyTuple_New(2 * (want[0] + want[1]));
    if (!r) return nullptr;
    for (int i = 0, k = 0; i < 4; ++i) {
        if (!want[i / 2]) continue;
        if (!made[i].defined()) changed({m[i].t});
        PyTuple_SET_ITEM(r, k++, result(made[i], arg[7 + i]));
    }
    return r;
    END_HANDLE_TH_ERRORS
}

// linear_fp8(x, x_scale, w, w_scale, bias, activation, residual, preact, out, dtype, workspace, stream) -> out
PyObject *linear_fp8(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 12)) return nullptr;
    Common all;
    Matrix x, xs, w, ws, r, z, y;
    Vector b;
    if (!x.read(all, arg[0], "x", true) || !xs.read(all, arg[1], "x_scale", true) || !w.read(all, arg[2], "w", true) ||
        !ws.read(all, arg[3], "w_scale", true) || !b.read(all, arg[4], "bias", w.d.rows) ||
        !r.read(all, arg[6], "residual", false) || !z.read(all, arg[7], "preact", false) ||
        !y.read(all, arg[8], "out", false) || !Workspace::admit(all, arg[10]))
        return nullptr;
    conv_linear_params p{};
    if (!activation_code(arg[5], &p.activation)) return nullptr;
    if (p.activation < 0) return status(CONV_ERR_BAD_PARAM);
    p.bias_dtype = b.type;
    at::ScalarType type;
    if (!scalar_type(arg[9], &type)) return nullptr;
    const Call c(*x.t, arg[11]);
    at::Tensor made;
    if (!y.t) {
        at::DimVector sizes(x.t->sizes().begin(), x.t->sizes().end());
        sizes.back() = w.d.rows;
        made = c.empty(sizes, type);
        if (!y.read(made, "out")) return nullptr;
    }
    size_t need = 0;
    conv_status st = conv_linear_fp8_workspace_size(&x.d, x.p, &w.d, w.p, &need);
    if (st) return status(st);
    Workspace work;
    if (!work.take(all, c, arg[10], need)) return nullptr;
    st = conv_linear_fp8(&x.d, x.p, &xs.d, xs.p, &w.d, w.p, &ws.d, ws.p, b.p, r.desc(), r.p, z.desc(), z.p, &y.d, y.p, &p,
                         work.p, work.bytes, c.stream);
    if (st) return status(st);
    if (made.defined()) y.t = nullptr;
    changed({z.t, y.t});
    return result(made, arg[8]);
    END_HANDLE_TH_ERRORS
}

// block_norm(x, skip, post_norm, post_gain, gate, skip_scale, branch_scale, gain, norm, eps, sum, out, out_scale, dtype,
//            post_rstd, rstd, stream) -> (sum or None, out or None[, out_scale])
PyObject *block_norm(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 17)) return nullptr;
    Common all;
    Matrix x, skip, gate, sum, y, ys;
    Vector pg, g, prstd, rstd;
    if (!x.read(all, arg[0], "x", true) || !skip.read(all, arg[1], "skip", false) ||
        !pg.read(all, arg[3], "post_gain", x.d.cols) || !gate.read(all, arg[4], "gate", false) ||
        !g.read(all, arg[7], "gain", x.d.cols) || !sum.read(all, arg[10], "sum", false) ||
        !y.read(all, arg[11], "out", false) || !ys.read(all, arg[12], "out_scale", false) ||
        !prstd.read_float(all, arg[14], "post_rstd", x.d.rows) || !rstd.read_float(all, arg[15], "rstd", x.d.rows))
        return nullptr;
    conv_block_norm_params p{};
    p.post_norm = PyObject_IsTrue(arg[2]) == 1;
    const bool norm = PyObject_IsTrue(arg[8]) == 1;
    if (!number(arg[5], &p.skip_scale) || !number(arg[6], &p.branch_scale) || !number(arg[9], &p.eps)) return nullptr;
    if (!float_types({&pg, &g})) return status(CONV_ERR_DTYPE);
    if (!one_type({&pg, &g}, &p.param_dtype)) return nullptr;
    at::ScalarType type = x.t->scalar_type();
    if (arg[13] != Py_None && !scalar_type(arg[13], &type)) return nullptr;
    if (!norm && (y.t || ys.t || rstd.t)) {
        PyErr_SetString(PyExc_ValueError, "out, out_scale and rstd belong to the norm, which is not wanted");
        return nullptr;
    }
    if (!p.post_norm && (pg.t || prstd.t)) {
        PyErr_SetString(PyExc_ValueError, "post_gain and post_rstd belong to the post norm, which is not wanted");
        return nullptr;
    }
    const Call c(*x.t, arg[16]);
    at::Tensor made_sum, made, made_scale;
    // (without any of these the sum is x itself)
    if (!sum.t && (skip.t || gate.t || p.post_norm || p.branch_scale != 1.0f || !norm)) {
        made_sum = c.empty(x.t->sizes(), skip.t ? skip.t->scalar_type() : x.t->scalar_type());
        if (!sum.read(made_sum, "sum")) return nullptr;
    }
    bool eight = false;
    if (norm) {
        if (!y.t) {
            made = type == at::kFloat8_e4m3fn ? eight_bit_for(c, x.t, x.d.rows, x.d.cols, type) : c.empty(x.t->sizes(), type);
            if (!y.read(made, "out")) return nullptr;
        }
        eight = y.d.dtype == CONV_FLOAT8_E4M3;
        if (!eight && ys.t) {
            PyErr_SetString(PyExc_ValueError, "out_scale belongs to an 8-bit out");
            return nullptr;
        }
        if (eight && !ys.t) {
            made_scale = scales_for(c, x.t, x.d.rows, x.d.cols, 1);
            if (!ys.read(made_scale, "out_scale")) return nullptr;
        }
    }
    const conv_status st = conv_block_norm(&x.d, x.p, skip.desc(), skip.p, gate.desc(), gate.p, pg.p, g.p, sum.desc(), sum.p,
                                           y.desc(), y.p, ys.desc(), ys.p, (float *)prstd.p, (float *)rstd.p, &p, c.stream);
    if (st) return status(st);
    if (!made_sum.defined()) changed({sum.t});
    if (!made.defined()) changed({y.t});
    if (!made_scale.defined()) changed({ys.t});
    changed({prstd.t, rstd.t});
    PyObject *r = PyTuple_New(eight ? 3 : 2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, result(made_sum, arg[10]));
    PyTuple_SET_ITEM(r, 1, result(made, arg[11]));
    if (eight) PyTuple_SET_ITEM(r, 2, result(made_scale, arg[12]));
    return r;
    END_HANDLE_TH_ERRORS
}

// block_norm_grad(dy, dsum, x, sum, post_norm, post_gain, gate, skip_scale, branch_scale, gain, post_rstd, rstd,
//                 dx, dskip, dgate, dgain, dpost_gain, workspace, stream) -> None
PyObject *block_norm_grad(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 19)) return nullptr;
    Common all;
    Matrix dy, ds, x, h, gate, dx, dskip, dgate;
    Vector pg, g, prstd, rstd, dg, dpg;
    if (!dy.read(all, arg[0], "dy", false) || !ds.read(all, arg[1], "dsum", false)) return nullptr;
    if (!dy.t && !ds.t) {
        PyErr_SetString(PyExc_ValueError, "dy or dsum is required");
        return nullptr;
    }
    const Matrix &like = dy.t ? dy : ds;
    const int64_t rows = like.d.rows, cols = like.d.cols;
    if (!x.read(all, arg[2], "x", false) || !h.read(all, arg[3], "sum", false) || !pg.read(all, arg[5], "post_gain", cols) ||
        !gate.read(all, arg[6], "gate", false) || !g.read(all, arg[9], "gain", cols) ||
        !prstd.read_float(all, arg[10], "post_rstd", rows) || !rstd.read_float(all, arg[11], "rstd", rows) ||
        !dx.read(all, arg[12], "dx", false) || !dskip.read(all, arg[13], "dskip", false) ||
        !dgate.read(all, arg[14], "dgate", false) || !dg.read(all, arg[15], "dgain", cols) ||
        !dpg.read(all, arg[16], "dpost_gain", cols) || !Workspace::admit(all, arg[17]))
        return nullptr;
    conv_block_norm_params p{};
    p.eps = 1e-6f;  // (in the statistics already)
    p.post_norm = PyObject_IsTrue(arg[4]) == 1;
    if (!number(arg[7], &p.skip_scale) || !number(arg[8], &p.branch_scale)) return nullptr;
    if (!float_types({&pg, &g, &dg, &dpg})) return status(CONV_ERR_DTYPE);
    if (!one_type({&pg, &g, &dg, &dpg}, &p.param_dtype)) return nullptr;
    const Call c(*like.t, arg[18]);
    const int64_t groups = gate.t ? gate.d.rows : dgate.t ? dgate.d.rows : rows > 0 ? 1 : 0;
    size_t need = 0;
    conv_status st = conv_block_norm_grad_workspace_size(&like.d, groups, &need);
    if (st) return status(st);
    Workspace ws;
    if (!ws.take(all, c, arg[17], need)) return nullptr;
    st = conv_block_norm_grad(dy.desc(), dy.p, ds.desc(), ds.p, x.desc(), x.p, h.desc(), h.p, gate.desc(), gate.p, pg.p, g.p,
                              (const float *)prstd.p, (const float *)rstd.p, dx.desc(), dx.p, dskip.desc(), dskip.p,
                              dgate.desc(), dgate.p, dpg.p, dg.p, &p, ws.p, ws.bytes, c.stream);
    if (st) return status(st);
    changed({dx.t, dskip.t, dgate.t, dg.t, dpg.t});
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// clip_grads(grads, max_norm, eps, out, norm, workspace, stream) -> norm
PyObject *clip_grads(PyObject *, PyObject *const *arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!count(n, 7)) return nullptr;
    Common all;
    struct Items {
        PyObject *o = nullptr;
        ~Items() { Py_XDECREF(o); }
    } grads, outs;
    grads.o = PySequence_Fast(arg[0], "grads must be a sequence of tensors");
    if (!grads.o) return nullptr;
    if (arg[3] != Py_None && !(outs.o = PySequence_Fast(arg[3], "out must be a sequence of tensors"))) return nullptr;
    const Py_ssize_t k = PySequence_Fast_GET_SIZE(grads.o);
    if (outs.o && PySequence_Fast_GET_SIZE(outs.o) != k) {
        PyErr_SetString(PyExc_ValueError, "out must have a tensor for every one of grads");
        return nullptr;
    }
    std::vector<conv_grad_tensor> table((size_t)k);
    std::vector<const at::Tensor *> written((size_t)k);
    for (Py_ssize_t i = 0; i < k; ++i) {
        bool ok;
        const at::Tensor *g = tensor(all, PySequence_Fast_GET_ITEM(grads.o, i), "a gradient", &ok);
        if (!ok) return nullptr;
        const at::Tensor *o = g;
        if (!g) return fail("a gradient", "is None; leave it out"), nullptr;
        if (!g->is_non_overlapping_and_dense()) return fail("a gradient", "has gaps between its elements; make it contiguous"), nullptr;
        if (outs.o) {
            o = tensor(all, PySequence_Fast_GET_ITEM(outs.o, i), "an out", &ok);
            if (!ok) return nullptr;
            if (!o) return fail("an out", "is None"), nullptr;
            if (o->scalar_type() != g->scalar_type() || o->sizes() != g->sizes() || o->strides() != g->strides())
                return fail("an out", "must have its gradient's type, shape and strides"), nullptr;
        }
        table[i] = {g->numel() ? g->data_ptr() : nullptr, o->numel() ? o->data_ptr() : nullptr, g->numel(), type_code(g->scalar_type()), 0};
        written[i] = o;
    }
    float max_norm, eps;
    if (!number(arg[1], &max_norm) || !number(arg[2], &eps)) return nullptr;
    if (outs.o && std::isinf(max_norm))  // (the library would leave them as they are)
        return fail("out", "is for clipped tensors; without a finite max_norm nothing is clipped"), nullptr;
    bool ok;
    const at::Tensor *norm = tensor(all, arg[4], "norm", &ok);
    if (!ok || !Workspace::admit(all, arg[5])) return nullptr;
    if (norm && (norm->numel() != 1 || norm->scalar_type() != at::kFloat)) return fail("norm", "must be one float32"), nullptr;
    if (!all.first) return fail("grads", "has no tensors; without them norm is required"), nullptr;
    const Call c(*all.first, arg[6]);
    at::Tensor made;
    if (!norm) made = c.empty({}, at::kFloat);
    size_t need = 0;
    conv_status st = conv_clip_grads_workspace_size(table.data(), k, &need);
    if (st) return status(st);
    Workspace ws;
    if (!ws.take(all, c, arg[5], need)) return nullptr;
    st = conv_clip_grads(table.data(), k, max_norm, eps, (float *)(norm ? norm->data_ptr() : made.data_ptr()), ws.p, ws.bytes, c.stream);
    if (st) return status(st);
    if (!std::isinf(max_norm))
        for (const at::Tensor *t : written) changed({t});
    changed({norm});
    return result(made, arg[4]);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"quantize", (PyCFunction)(void (*)())quantize, METH_FASTCALL, nullptr},
    {"linear_fp8", (PyCFunction)(void (*)())linear_fp8, METH_FASTCALL, nullptr},
    {"block_norm", (PyCFunction)(void (*)())block_norm, METH_FASTCALL, nullptr},
    {"block_norm_grad", (PyCFunction)(void (*)())block_norm_grad, METH_FASTCALL, nullptr},
    {"clip_grads", (PyCFunction)(void (*)())clip_grads, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void (*)())linear, METH_FASTCALL, nullptr},
    {"linear_grad", (PyCFunction)(void (*)())linear_grad, METH_FASTCALL, nullptr},
    {"layer_norm", (PyCFunction)(void (*)())layer_norm, METH_FASTCALL, nullptr},
    {"layer_norm_grad", (PyCFunction)(void (*)())layer_norm_grad, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_channel", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__channel(void) { return PyModule_Create(&module); }
