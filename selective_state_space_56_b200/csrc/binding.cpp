// binding.cpp -- native marshalling for the layer operators' calls.
//
// A decode step's kernels take 3 to 8 us; checking a handful of tensors and allocating the outputs
// through the interpreter took 5 to 10 us a call on top of the launch.  These functions do the same
// checks and allocations on the C++ side of torch and forward to the same C entry points, whose
// addresses ops.py hands over (bind).  Whatever is not plainly in order -- another dtype, shape,
// device or layout -- makes them return None before anything is called, and ops.py's own path
// then finds out what is wrong and says so.  Once the library has been called there is no second
// call (the update works in place): a status other than MAMBA_OK is raised as MambaError, and so is
// whatever else goes wrong from there on.  No arithmetic, no state but the addresses and that class.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mamba_s6.h"

namespace {

#define CALLS(X)                                                                                   \
    X(mamba_gated_scan_fwd) X(mamba_gated_scan_bwd) X(mamba_gated_state_update)                     \
    X(mamba_gated_scan_bwd_workspace_size) X(mamba_add_rms_norm_fwd) X(mamba_add_rms_norm_fp8)      \
    X(mamba_add_rms_norm_bwd) X(mamba_add_rms_norm_bwd_workspace_size) X(mamba_fp8_quantize)        \
    X(mamba_fp8_linear)

struct Calls {
#define X(name) decltype(&::name) name = nullptr;
    CALLS(X)
#undef X
};
Calls calls;
bool bound = false;
PyObject* error_class = nullptr;  // ops.MambaError(status, name of the call)

constexpr at::ScalarType kF32 = at::kFloat, kE4m3 = at::kFloat8_e4m3fn;

// The library's code of a dtype it takes, or -1.
int code_of(at::ScalarType t) { return t == at::kFloat ? MAMBA_F32 : t == at::kBFloat16 ? MAMBA_BF16 : -1; }

// The arguments of one call: every check notes a failure, and the call is made if there was none.
struct Args {
    int dev = -1;
    bool ok = true;

    const at::Tensor* plain(PyObject* o) {
        if (!THPVariable_CheckExact(o)) return ok = false, nullptr;
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided || !t.is_cuda() || !t.is_contiguous()) return ok = false, nullptr;
        return &t;
    }
    // The tensor that sets the device, which has to be the current one.
    const at::Tensor* first(PyObject* o) {
        const at::Tensor* t = plain(o);
        if (!t) return nullptr;
        dev = t->get_device();
        if (c10::cuda::current_device() != dev) return ok = false, nullptr;
        return t;
    }
    void* address(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape) {
        const at::Tensor* t = plain(o);
        if (!t) return nullptr;
        if (t->get_device() != dev || t->scalar_type() != dtype || t->sizes() != shape) return ok = false, nullptr;
        return t->data_ptr();
    }
    void* maybe(PyObject* o, at::ScalarType dtype, at::IntArrayRef shape) {
        return o == Py_None ? nullptr : address(o, dtype, shape);
    }
    // A caller's buffer of any dtype and shape.
    void* buffer(PyObject* o, size_t* bytes) {
        *bytes = 0;
        if (o == Py_None) return nullptr;
        const at::Tensor* t = plain(o);
        if (!t || t->get_device() != dev) return ok = false, nullptr;
        *bytes = t->nbytes();
        return t->data_ptr();
    }
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
        return at::detail::empty_cuda(shape, dtype, at::Device(at::kCUDA, (c10::DeviceIndex)dev), std::nullopt);
    }
    void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

float* f32(void* p) { return static_cast<float*>(p); }
PyObject* none() { Py_RETURN_NONE; }

// A call of the library without the interpreter's lock, as ctypes makes it: a launch can wait for room in
// the launch queue, and what makes room (a host function on a stream, another thread) may need the lock.
template <typename F>
int unlocked(F call) {
    struct Unlock {
        PyThreadState* thread = PyEval_SaveThread();
        ~Unlock() { PyEval_RestoreThread(thread); }
    } unlock;
    return call();
}

// What follows runs after the library's call and so reports its failures as exceptions.
PyObject* failed(int status, const char* name) {
    PyObject* e = PyObject_CallFunction(error_class, "is", status, name);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return nullptr;
}
PyObject* wrap(const at::Tensor& t) noexcept {
    PyObject* o = nullptr;
    try {
        o = THPVariable_Wrap(t);
    } catch (...) {
    }
    if (!o && !PyErr_Occurred()) PyErr_NoMemory();
    return o;
}
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    bool whole = r != nullptr;
    for (PyObject* o : items) {
        if (!o) whole = false;
        if (r) PyTuple_SET_ITEM(r, i, o);
        else Py_XDECREF(o);
        ++i;
    }
    if (whole) return r;
    Py_XDECREF(r);
    return nullptr;
}
PyObject* or_none(const at::Tensor& t) { return t.defined() ? wrap(t) : none(); }

// (state, x, gate, gate_bias, z, flags) -> y
PyObject* gated_state_update(PyObject* const* o) {
    Args a;
    const at::Tensor *s = a.first(o[0]), *x = a.plain(o[1]);
    if (!a.ok || s->dim() != 2 || s->scalar_type() != kF32) return none();
    const unsigned flags = (unsigned)PyLong_AsLong(o[5]);
    const auto shape = s->sizes();
    const auto dt = x->scalar_type();
    const int code = code_of(dt);
    void *xp = a.address(o[1], dt, shape), *g = a.address(o[2], dt, shape), *b = a.maybe(o[3], kF32, shape[1]),
         *z = a.maybe(o[4], dt, shape);
    if (!a.ok || code < 0) return none();
    const at::Tensor y = a.empty(shape, dt);
    const int rc = unlocked([&] {
        return calls.mamba_gated_state_update(f32(s->data_ptr()), xp, g, f32(b), z, y.data_ptr(), shape[0], shape[1],
                                              (mamba_dtype)code, flags, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_gated_state_update");
    return wrap(y);
}

// (x, gate, gate_bias, z, initial_state, checkpoints, flags, want last_state) -> (y, last_state or None)
PyObject* gated_scan_fwd(PyObject* const* o) {
    Args a;
    const at::Tensor* x = a.first(o[0]);
    if (!a.ok || x->dim() != 3) return none();
    const auto shape = x->sizes();
    const auto dt = x->scalar_type();
    const int code = code_of(dt);
    const unsigned flags = (unsigned)PyLong_AsLong(o[6]);
    const int64_t rows[2] = {shape[0], shape[1]};
    void *g = a.address(o[1], dt, shape), *b = a.maybe(o[2], kF32, shape[1]), *z = a.maybe(o[3], dt, shape),
         *h0 = a.maybe(o[4], kF32, rows);
    size_t ck_bytes;
    void* ck = a.buffer(o[5], &ck_bytes);
    if (!a.ok || code < 0) return none();
    const at::Tensor y = a.empty(shape, dt);
    at::Tensor last;
    if (o[7] == Py_True) last = a.empty(rows, kF32);
    const int rc = unlocked([&] {
        return calls.mamba_gated_scan_fwd(x->data_ptr(), g, f32(b), z, f32(h0), y.data_ptr(),
                                          last.defined() ? f32(last.data_ptr()) : nullptr, f32(ck), ck_bytes,
                                          {shape[0], shape[1], shape[2]}, (mamba_dtype)code, (mamba_dtype)code,
                                          flags, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_gated_scan_fwd");
    return tuple({wrap(y), or_none(last)});
}

// (x, gate, dy, gate_bias, z, initial_state, dlast_state, checkpoints, flags)
// -> (dx, dgate, dz or None, dgate_bias or None, dinitial_state)
PyObject* gated_scan_bwd(PyObject* const* o) {
    Args a;
    const at::Tensor* x = a.first(o[0]);
    if (!a.ok || x->dim() != 3) return none();
    const auto shape = x->sizes();
    const auto dt = x->scalar_type();
    const int code = code_of(dt);
    const int64_t rows[2] = {shape[0], shape[1]};
    const unsigned flags = (unsigned)PyLong_AsLong(o[8]);
    void *g = a.address(o[1], dt, shape), *dy = a.address(o[2], dt, shape), *b = a.maybe(o[3], kF32, shape[1]),
         *z = a.maybe(o[4], dt, shape), *h0 = a.maybe(o[5], kF32, rows), *dl = a.maybe(o[6], kF32, rows);
    size_t ck_bytes;
    void* ck = a.buffer(o[7], &ck_bytes);
    if (!a.ok || code < 0) return none();
    const mamba_gated_dims dims{shape[0], shape[1], shape[2]};
    const int64_t need = (int64_t)calls.mamba_gated_scan_bwd_workspace_size(dims);
    const at::Tensor dx = a.empty(shape, dt), dg = a.empty(shape, dt), dh0 = a.empty(rows, kF32);
    at::Tensor dz, db, ws;
    if (o[4] != Py_None) dz = a.empty(shape, dt);  // (the address of a z without elements is null)
    if (b && !(flags & MAMBA_FLAG_GIVEN_DECAY)) db = a.empty(shape[1], kF32);
    if (need > 0) ws = a.empty(need, at::kByte);
    const int rc = unlocked([&] {
        return calls.mamba_gated_scan_bwd(x->data_ptr(), g, f32(b), z, f32(h0), dy, f32(dl), dx.data_ptr(), dg.data_ptr(),
                                          dz.defined() ? dz.data_ptr() : nullptr, db.defined() ? f32(db.data_ptr()) : nullptr,
                                          f32(dh0.data_ptr()), f32(ck), ck_bytes, dims, (mamba_dtype)code,
                                          need > 0 ? ws.data_ptr() : nullptr, (size_t)need, flags, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_gated_scan_bwd");
    return tuple({wrap(dx), wrap(dg), or_none(dz), or_none(db), wrap(dh0)});
}

// x, weight and residual of a norm: rows, dim, dtypes and addresses.
struct Norm {
    const at::Tensor* x = nullptr;
    at::IntArrayRef shape;
    int64_t rows = 0, dim = 0;
    at::ScalarType dt, rt;
    int code = -1, rcode = -1;
    void *weight = nullptr, *residual = nullptr;

    Norm(Args& a, PyObject* xo, PyObject* wo, PyObject* ro) : dt(kF32), rt(kF32) {
        x = a.first(xo);
        if (!a.ok || x->dim() < 2 || x->dim() > 3) {
            a.ok = false;
            return;
        }
        shape = x->sizes();
        dim = shape.back();
        rows = shape.size() == 2 ? shape[0] : shape[0] * shape[1];
        dt = rt = x->scalar_type();
        if (ro != Py_None) {
            const at::Tensor* r = a.plain(ro);
            if (!r) return;
            rt = r->scalar_type();
            residual = a.address(ro, rt, shape);
        }
        code = code_of(dt), rcode = code_of(rt);
        weight = a.address(wo, kF32, dim);
        if (code < 0 || rcode < 0) a.ok = false;
    }
};

// (x, weight, residual, eps) -> (out, residual_out or None)
PyObject* add_rms_norm_fwd(PyObject* const* o) {
    Args a;
    const Norm n(a, o[0], o[1], o[2]);
    const double eps = PyFloat_Check(o[3]) ? PyFloat_AS_DOUBLE(o[3]) : (a.ok = false, 0.0);
    if (!a.ok) return none();
    const at::Tensor out = a.empty(n.shape, n.dt);
    at::Tensor v;
    if (o[2] != Py_None) v = a.empty(n.shape, n.rt);
    const int rc = unlocked([&] {
        return calls.mamba_add_rms_norm_fwd(n.x->data_ptr(), n.residual, f32(n.weight), (float)eps, out.data_ptr(),
                                            v.defined() ? v.data_ptr() : nullptr, n.rows, n.dim, (mamba_dtype)n.code,
                                            (mamba_dtype)n.rcode, (mamba_dtype)n.code, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_add_rms_norm_fwd");
    return tuple({wrap(out), or_none(v)});
}

// (x, weight, residual, eps) -> (q, scales, residual_out or None)
PyObject* add_rms_norm_fp8(PyObject* const* o) {
    Args a;
    const Norm n(a, o[0], o[1], o[2]);
    const double eps = PyFloat_Check(o[3]) ? PyFloat_AS_DOUBLE(o[3]) : (a.ok = false, 0.0);
    if (!a.ok) return none();
    int64_t groups[3];
    for (size_t i = 0; i < n.shape.size(); ++i) groups[i] = n.shape[i];
    groups[n.shape.size() - 1] = (n.dim + 127) / 128;
    const at::Tensor q = a.empty(n.shape, kE4m3), s = a.empty(at::IntArrayRef(groups, n.shape.size()), kF32);
    at::Tensor v;
    if (o[2] != Py_None) v = a.empty(n.shape, n.rt);
    const int rc = unlocked([&] {
        return calls.mamba_add_rms_norm_fp8(n.x->data_ptr(), n.residual, f32(n.weight), (float)eps, q.data_ptr(),
                                            f32(s.data_ptr()), v.defined() ? v.data_ptr() : nullptr, n.rows, n.dim,
                                            (mamba_dtype)n.code, (mamba_dtype)n.rcode, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_add_rms_norm_fp8");
    return tuple({wrap(q), wrap(s), or_none(v)});
}

// (dout, residual_out, weight, dresidual_out, eps) -> (dx, dresidual or None where dx serves, dweight)
PyObject* add_rms_norm_bwd(PyObject* const* o) {
    Args a;
    const Norm n(a, o[0], o[2], o[1]);
    const double eps = PyFloat_Check(o[4]) ? PyFloat_AS_DOUBLE(o[4]) : (a.ok = false, 0.0);
    if (!a.ok || o[1] == Py_None) return none();
    void* ds = a.maybe(o[3], n.rt, n.shape);
    if (!a.ok) return none();
    const int64_t need = (int64_t)calls.mamba_add_rms_norm_bwd_workspace_size(n.rows, n.dim);
    const at::Tensor dx = a.empty(n.shape, n.dt), dw = a.empty(n.dim, kF32);
    at::Tensor dres, ws;
    if (n.rt != n.dt) dres = a.empty(n.shape, n.rt);
    if (need > 0) ws = a.empty(need, at::kByte);
    const int rc = unlocked([&] {
        return calls.mamba_add_rms_norm_bwd(n.x->data_ptr(), n.residual, f32(n.weight), ds, (float)eps, dx.data_ptr(),
                                            dres.defined() ? dres.data_ptr() : nullptr, f32(dw.data_ptr()), n.rows, n.dim,
                                            (mamba_dtype)n.code, (mamba_dtype)n.rcode, need > 0 ? ws.data_ptr() : nullptr,
                                            (size_t)need, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_add_rms_norm_bwd");
    return tuple({wrap(dx), or_none(dres), wrap(dw)});
}

// (x, channel_major) -> (q, scales)
PyObject* fp8_quantize(PyObject* const* o) {
    Args a;
    const at::Tensor* x = a.first(o[0]);
    const bool cm = o[1] == Py_True;
    if (!a.ok || x->dim() != (cm ? 3 : 2)) return none();
    const int code = code_of(x->scalar_type());
    if (code < 0) return none();
    const auto in = x->sizes();
    const int64_t b = cm ? in[0] : 1, d = in[1], len = cm ? in[2] : in[0];
    const int64_t qs[2] = {b * len, d}, ss[2] = {b * len, (d + 127) / 128};
    const at::Tensor q = a.empty(qs, kE4m3), s = a.empty(ss, kF32);
    const int rc = unlocked([&] {
        return calls.mamba_fp8_quantize(x->data_ptr(), q.data_ptr(), f32(s.data_ptr()), b, d, len, cm ? 1 : 0,
                                        (mamba_dtype)code, a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_fp8_quantize");
    return tuple({wrap(q), wrap(s)});
}

// (xq, x_scales, wq, w_scales, code of the output's dtype, L or 0) -> out
PyObject* fp8_linear(PyObject* const* o) {
    Args a;
    const at::Tensor *x = a.first(o[0]), *w = a.plain(o[2]);
    const long code = PyLong_AsLong(o[4]), len = PyLong_AsLong(o[5]);
    if (!a.ok || x->dim() != 2 || w->dim() != 2 || len < 0) return none();
    const int64_t t = x->size(0), k = x->size(1), n = w->size(0), kb = (k + 127) / 128;
    const int64_t xs_shape[2] = {t, kb}, w_shape[2] = {n, k}, ws_shape[2] = {(n + 127) / 128, kb};
    void *xs = a.address(o[1], kF32, xs_shape), *wp = a.address(o[2], kE4m3, w_shape),
         *ws = a.address(o[3], kF32, ws_shape);
    if (!a.ok || x->scalar_type() != kE4m3 || (code != MAMBA_F32 && code != MAMBA_BF16) || (len > 0 && t % len != 0))
        return none();
    const at::ScalarType dt = code == MAMBA_F32 ? at::kFloat : at::kBFloat16;
    const int64_t rows[2] = {t, n}, cols[3] = {len > 0 ? t / len : 0, n, len};
    const at::Tensor out = len > 0 ? a.empty(cols, dt) : a.empty(rows, dt);
    const int rc = unlocked([&] {
        return calls.mamba_fp8_linear(x->data_ptr(), f32(xs), wp, f32(ws), out.data_ptr(), t, n, k, len, (mamba_dtype)code,
                                      a.stream());
    });
    if (rc != MAMBA_OK) return failed(rc, "mamba_fp8_linear");
    return wrap(out);
}

// Number of arguments, nothing thrown past the interpreter's boundary.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N || !bound || !error_class) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or called before bind() and set_error()");
        return nullptr;
    }
    try {
        return F(args);
    } catch (...) {  // checks and allocations, before the call
        PyErr_Clear();
        return none();
    }
}

// bind({name: address}): the C entry points.
PyObject* bind(PyObject*, PyObject* names) {
#define X(name)                                                                            \
    {                                                                                      \
        PyObject* v = PyDict_Check(names) ? PyDict_GetItemString(names, #name) : nullptr;  \
        void* p = v ? PyLong_AsVoidPtr(v) : nullptr;                                       \
        if (!p) {                                                                          \
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #name);                 \
            return nullptr;                                                                \
        }                                                                                  \
        calls.name = reinterpret_cast<decltype(calls.name)>(p);                            \
    }
    CALLS(X)
#undef X
    bound = true;
    Py_RETURN_NONE;
}

// set_error(class): what a failed call raises, made from its status and its name.
PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(error_class, cls);
    Py_RETURN_NONE;
}

PyObject* names(PyObject*, PyObject*) {
    PyObject* r = PyList_New(0);
#define X(name)                                                 \
    {                                                           \
        PyObject* s = PyUnicode_FromString(#name);              \
        if (r && s) PyList_Append(r, s);                        \
        Py_XDECREF(s);                                          \
    }
    CALLS(X)
#undef X
    return r;
}

#define FAST(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"bind", bind, METH_O, nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {"names", names, METH_NOARGS, nullptr},
                         FAST(gated_state_update, 6),
                         FAST(gated_scan_fwd, 8),
                         FAST(gated_scan_bwd, 9),
                         FAST(add_rms_norm_fwd, 4),
                         FAST(add_rms_norm_fp8, 4),
                         FAST(add_rms_norm_bwd, 5),
                         FAST(fp8_quantize, 2),
                         FAST(fp8_linear, 6),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) {
    PyObject* m = PyModule_Create(&module);
    // the torch it was compiled against: ops.py uses it with that one only
    if (m && PyModule_AddStringConstant(m, "torch_version", S6_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
