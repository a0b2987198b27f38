// Argument marshalling of small calls: the same C entry points as the ctypes
// binding's (layer_ops.py), reached from tensors in one C call.  A call of one
// token lasts a few microseconds on the GPU and, through ctypes, 15 on the host:
// most of it Python's attribute and allocation calls.
//
// Each function answers plain calls (tensors of expected types and shapes on the
// current device, outputs and workspace to be allocated) and returns None for any
// other, which the Python code then takes: every refusal, message and further
// layout is decided there.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <climits>

#include "ssd.h"

namespace {

// A tensor argument, or nullptr for None (ok stays true) and for anything that is
// not a contiguous CUDA tensor on `device` (ok becomes false; device < 0: any) or
// whose dimensions pass the C interface's ints.
const at::Tensor *tensor(PyObject *o, int device, bool &ok) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
        ok = false;
        return nullptr;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.is_contiguous() || t.dim() < 1 || t.numel() == 0 ||
        t.size(0) > INT_MAX || t.size(-1) > INT_MAX ||
        (device >= 0 && t.get_device() != device)) {
        ok = false;
        return nullptr;
    }
    return &t;
}

// The same for a matrix whose rows lie at one stride of at least their width.
struct Matrix {
    const at::Tensor *t = nullptr;
    int64_t stride = 0;
};
Matrix matrix(PyObject *o, int device, bool &ok) {
    Matrix m;
    if (o == Py_None) return m;
    if (!THPVariable_Check(o)) {
        ok = false;
        return m;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() < 2 || t.numel() == 0 || t.size(-1) > INT_MAX ||
        (t.size(-1) > 1 && t.stride(-1) != 1) || (device >= 0 && t.get_device() != device)) {
        ok = false;
        return m;
    }
    int64_t row = -1, step = 0;
    for (int64_t d = t.dim() - 2; d >= 0; --d) {
        if (t.size(d) == 1) continue;
        if (row < 0) row = t.stride(d);
        else if (t.stride(d) != step) ok = false;
        step = t.stride(d) * t.size(d);
    }
    m.t = &t;
    m.stride = row < 0 ? t.size(-1) : row;
    if (m.stride < t.size(-1)) ok = false;
    return m;
}
bool like(const Matrix &m, const at::Tensor &x) {
    return !m.t || (m.t->sizes() == x.sizes() && m.t->scalar_type() == x.scalar_type());
}

int code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return SSD_F32;
        case at::kBFloat16: return SSD_BF16;
        case at::ScalarType::Float8_e4m3fn: return SSD_FP8_E4M3;
        default: return -1;
    }
}
at::ScalarType type_of(int code) {
    return code == SSD_F32 ? at::kFloat
                           : (code == SSD_BF16 ? at::kBFloat16 : at::ScalarType::Float8_e4m3fn);
}

bool vector(const at::Tensor *t, int64_t n) {
    return !t || (t->scalar_type() == at::kFloat && t->dim() == 1 && t->size(0) == n);
}
bool floats(const at::Tensor *t, int64_t n) {
    return !t || (t->scalar_type() == at::kFloat && t->numel() == n);
}

const void *ptr(const at::Tensor *t) { return t ? t->const_data_ptr() : nullptr; }
const float *fptr(const at::Tensor *t) { return t ? t->const_data_ptr<float>() : nullptr; }

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// The status as an int for Python to raise on, or the answer.
PyObject *answer(ssd_status st, PyObject *value) {
    if (st == SSD_OK) return value;
    Py_XDECREF(value);
    return PyLong_FromLong((long)st);
}

// x, weight, residual or None, eps, out code -> (y, residual_out or None, rstd, scale or None)
PyObject *rmsnorm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 5;
    const at::Tensor *x = ok ? tensor(args[0], -1, ok) : nullptr;
    if (!x || x->dim() < 2 || x->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x->get_device();
    const at::Tensor *w = tensor(args[1], dev, ok), *r = tensor(args[2], dev, ok);
    const double eps = PyFloat_AsDouble(args[3]);
    const int out = (int)PyLong_AsLong(args[4]), xc = code(x->scalar_type());
    const int64_t width = x->size(-1), rows = x->numel() / width;
    if (PyErr_Occurred()) return nullptr;
    if (!ok || !w || !vector(w, width) || xc < 0 || (r && r->sizes() != x->sizes()))
        Py_RETURN_NONE;
    const int rc = r ? code(r->scalar_type()) : xc;
    if (rc < 0) Py_RETURN_NONE;
    const auto lead = x->sizes().slice(0, x->dim() - 1);
    at::Tensor y = make(x->sizes(), type_of(out), *x), rstd = make(lead, at::kFloat, *x), so, scale;
    if (r) so = make(x->sizes(), r->scalar_type(), *x);
    if (out == SSD_FP8_E4M3) scale = make(lead, at::kFloat, *x);
    const ssd_status st = ssd_rmsnorm_fwd(
        ptr(x), ptr(r), fptr(w), (float)eps, (ssd_dtype)xc, (ssd_dtype)rc, (ssd_dtype)out, rows,
        (int)width, width, width, y.mutable_data_ptr(), r ? so.mutable_data_ptr() : nullptr,
        rstd.mutable_data_ptr<float>(), scale.defined() ? scale.mutable_data_ptr<float>() : nullptr,
        c10::cuda::getCurrentCUDAStream(dev));
    PyObject *t = PyTuple_New(4);
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(y));
    PyTuple_SET_ITEM(t, 1, r ? THPVariable_Wrap(so) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(rstd));
    PyTuple_SET_ITEM(t, 3, scale.defined() ? THPVariable_Wrap(scale) : Py_NewRef(Py_None));
    return answer(st, t);
    END_HANDLE_TH_ERRORS
}

// x, w, bias, residual, activation code, x_scale, w_scale, out code -> y
PyObject *linear_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 8;
    const at::Tensor *x = ok ? tensor(args[0], -1, ok) : nullptr;
    if (!x || x->dim() < 2 || x->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x->get_device();
    const at::Tensor *w = tensor(args[1], dev, ok), *b = tensor(args[2], dev, ok);
    const at::Tensor *r = tensor(args[3], dev, ok), *xs = tensor(args[5], dev, ok);
    const at::Tensor *ws = tensor(args[6], dev, ok);
    const int act = (int)PyLong_AsLong(args[4]), out = (int)PyLong_AsLong(args[7]);
    if (PyErr_Occurred()) return nullptr;
    if (!ok || !w || w->dim() != 2 || w->scalar_type() != x->scalar_type() ||
        w->size(1) != x->size(-1))
        Py_RETURN_NONE;
    const int xc = code(x->scalar_type());
    const int64_t inner = x->size(-1), tokens = x->numel() / inner, features = w->size(0);
    if (xc < 0 || !vector(b, features) || !vector(ws, features) || !floats(xs, tokens) ||
        (xs && xs->sizes() != x->sizes().slice(0, x->dim() - 1)))
        Py_RETURN_NONE;
    c10::SmallVector<int64_t, 6> shape(x->sizes().begin(), x->sizes().end());
    shape.back() = features;
    if (r && (r->scalar_type() != type_of(out) || r->sizes() != at::IntArrayRef(shape)))
        Py_RETURN_NONE;
    at::Tensor y = make(shape, type_of(out), *x);
    const ssd_status st = ssd_linear_fwd(
        ptr(x), fptr(xs), ptr(w), fptr(ws), fptr(b), ptr(r), (ssd_activation)act, (ssd_dtype)xc,
        (ssd_dtype)out, tokens, (int)features, (int)inner, inner, features, y.mutable_data_ptr(),
        features, nullptr, c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, THPVariable_Wrap(y));
    END_HANDLE_TH_ERRORS
}

// state, x, g, z or None -> y
PyObject *gated_state_update(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 4;
    const Matrix x = ok ? matrix(args[1], -1, ok) : Matrix();
    if (!ok || !x.t || x.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x.t->get_device();
    const Matrix g = matrix(args[2], dev, ok), z = matrix(args[3], dev, ok);
    const at::Tensor *state = tensor(args[0], dev, ok);
    const int c = code(x.t->scalar_type());
    if (!ok || !state || !g.t || !like(g, *x.t) || !like(z, *x.t) || c < 0 ||
        state->scalar_type() != at::kFloat || state->sizes() != x.t->sizes())
        Py_RETURN_NONE;
    const int64_t width = x.t->size(-1);
    at::Tensor y = make(x.t->sizes(), x.t->scalar_type(), *x.t);
    const ssd_status st = ssd_gated_state_update(
        state->mutable_data_ptr<float>(), ptr(x.t), ptr(g.t), ptr(z.t), (ssd_dtype)c,
        x.t->numel() / width, (int)width, x.stride, g.stride, z.stride, y.mutable_data_ptr(),
        c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, THPVariable_Wrap(y));
    END_HANDLE_TH_ERRORS
}

// A workspace of n bytes (undefined for 0).
at::Tensor scratch(size_t n, const at::Tensor &like) {
    return n ? make({(int64_t)n}, at::kByte, like) : at::Tensor();
}
PyObject *wrap(const at::Tensor &t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
PyObject *tuple4(PyObject *a, PyObject *b, PyObject *c, PyObject *d) {
    PyObject *t = PyTuple_New(4);
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    PyTuple_SET_ITEM(t, 2, c);
    PyTuple_SET_ITEM(t, 3, d);
    return t;
}
template <typename T = void>
T *out(at::Tensor &t) {
    return t.defined() ? static_cast<T *>(t.mutable_data_ptr()) : nullptr;
}

// dy, s, weight, rstd, dresidual -> (dx, ds (dx itself for one type), dweight, None)
PyObject *rmsnorm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 5;
    const Matrix dy = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !dy.t || dy.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = dy.t->get_device();
    const Matrix s = matrix(args[1], dev, ok), dr = matrix(args[4], dev, ok);
    const at::Tensor *w = tensor(args[2], dev, ok), *rstd = tensor(args[3], dev, ok);
    const int64_t width = dy.t->size(-1), rows = dy.t->numel() / width;
    const auto lead = dy.t->sizes().slice(0, dy.t->dim() - 1);
    if (!ok || !s.t || !w || !rstd || s.t->sizes() != dy.t->sizes() || !like(dr, *s.t) ||
        !vector(w, width) || rstd->scalar_type() != at::kFloat || rstd->sizes() != lead)
        Py_RETURN_NONE;
    const int c = code(dy.t->scalar_type()), sc = code(s.t->scalar_type());
    const size_t need = ssd_rmsnorm_bwd_workspace_bytes(rows, (int)width);
    if (c < 0 || sc < 0 || need == (size_t)-1) Py_RETURN_NONE;
    at::Tensor dx = make(dy.t->sizes(), dy.t->scalar_type(), *dy.t), ds;
    if (c != sc) ds = make(dy.t->sizes(), s.t->scalar_type(), *dy.t);
    at::Tensor dw = make({width}, at::kFloat, *dy.t), ws = scratch(need, *dy.t);
    const ssd_status st = ssd_rmsnorm_bwd(
        ptr(dy.t), ptr(s.t), fptr(w), fptr(rstd), ptr(dr.t), (ssd_dtype)c, (ssd_dtype)sc, rows,
        (int)width, dy.stride, s.stride, dr.stride, out(dx), out(ds), out<float>(dw), out(ws), need,
        c10::cuda::getCurrentCUDAStream(dev));
    PyObject *first = wrap(dx);
    return answer(st, tuple4(first, ds.defined() ? wrap(ds) : Py_NewRef(first), wrap(dw),
                             Py_NewRef(Py_None)));
    END_HANDLE_TH_ERRORS
}

// dy, x, w, preact, activation code, whether dbias is wanted -> (dx, dw, dbias or None, None)
PyObject *linear_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 6;
    const Matrix dy = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !dy.t || dy.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = dy.t->get_device();
    const Matrix x = matrix(args[1], dev, ok);
    const at::Tensor *w = tensor(args[2], dev, ok), *pre = tensor(args[3], dev, ok);
    const int act = (int)PyLong_AsLong(args[4]), bias = PyObject_IsTrue(args[5]);
    if (PyErr_Occurred()) return nullptr;
    const auto type = dy.t->scalar_type();
    if (!ok || !x.t || !w || w->dim() != 2 || x.t->scalar_type() != type ||
        w->scalar_type() != type || x.t->dim() != dy.t->dim())
        Py_RETURN_NONE;
    const int64_t features = dy.t->size(-1), tokens = dy.t->numel() / features;
    const int64_t inner = x.t->size(-1);
    if (w->size(0) != features || w->size(1) != inner ||
        x.t->sizes().slice(0, x.t->dim() - 1) != dy.t->sizes().slice(0, dy.t->dim() - 1) ||
        (pre && (pre->sizes() != dy.t->sizes() || pre->scalar_type() != type)))
        Py_RETURN_NONE;
    const int c = code(type);
    const size_t need = c < 0 ? (size_t)-1
                              : ssd_linear_bwd_workspace_bytes((ssd_dtype)c, (ssd_activation)act,
                                                               tokens, (int)features, (int)inner);
    if (need == (size_t)-1) Py_RETURN_NONE;
    at::Tensor dx = make(x.t->sizes(), type, *dy.t), dw = make({features, inner}, type, *dy.t), db;
    if (bias) db = make({features}, at::kFloat, *dy.t);
    at::Tensor ws = scratch(need, *dy.t);
    const ssd_status st = ssd_linear_bwd(
        ptr(dy.t), ptr(x.t), ptr(w), ptr(pre), (ssd_activation)act, (ssd_dtype)c, tokens,
        (int)features, (int)inner, dy.stride, x.stride, out(dx), out(dw), out<float>(db), out(ws),
        need, c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, tuple4(wrap(dx), wrap(dw), wrap(db), Py_NewRef(Py_None)));
    END_HANDLE_TH_ERRORS
}

// The sequences of a recurrence over x: [batch, length, width], or [tokens, width]
// with offsets as a list of ints and their device copy.
struct Sequences {
    int nseq = 0, length = 0;
    int64_t tokens = 0;
    c10::SmallVector<int, 64> host;
    const int *device = nullptr;
    const int *offsets() const { return host.empty() ? nullptr : host.data(); }
};
bool sequences(const at::Tensor &x, PyObject *cu, PyObject *cu_dev, Sequences &s) {
    s.tokens = x.numel() / x.size(-1);
    if (s.tokens > INT_MAX) return false;
    if (cu == Py_None) {
        if (x.dim() != 3) return false;
        s.nseq = (int)x.size(0);
        s.length = (int)x.size(1);
        return true;
    }
    bool ok = x.dim() == 2 && PyList_Check(cu) && PyList_GET_SIZE(cu) >= 2;
    const at::Tensor *d = ok ? tensor(cu_dev, x.get_device(), ok) : nullptr;
    if (!ok || !d || d->scalar_type() != at::kInt || d->dim() != 1 ||
        d->size(0) != PyList_GET_SIZE(cu))
        return false;
    for (Py_ssize_t i = 0; i < PyList_GET_SIZE(cu); ++i) {
        PyObject *v = PyList_GET_ITEM(cu, i);
        if (!PyLong_CheckExact(v)) return false;
        int over = 0;
        const long long o = PyLong_AsLongLongAndOverflow(v, &over);
        if (over || o < 0 || o > INT_MAX) return false;
        s.host.push_back((int)o);
    }
    s.nseq = (int)s.host.size() - 1;
    s.device = d->const_data_ptr<int>();
    return s.host.back() == s.tokens;
}

// x, g, z, init_state, offsets, device offsets, whether the checkpoints are wanted
// -> (y, final_state, checkpoints or None, None)
PyObject *gated_scan_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 7;
    const Matrix x = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !x.t || x.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x.t->get_device();
    const Matrix g = matrix(args[1], dev, ok), z = matrix(args[2], dev, ok);
    const at::Tensor *init = tensor(args[3], dev, ok);
    const int keep = PyObject_IsTrue(args[6]), c = code(x.t->scalar_type());
    if (keep < 0) return nullptr;       // no truth value: the exception is set
    Sequences q;
    if (!ok || !g.t || !like(g, *x.t) || !like(z, *x.t) || c < 0 ||
        !sequences(*x.t, args[4], args[5], q))
        Py_RETURN_NONE;
    const int64_t width = x.t->size(-1);
    const std::array<int64_t, 2> states{q.nseq, width};
    const size_t need = ssd_gated_scan_workspace_bytes((ssd_dtype)c, q.tokens, (int)width);
    if (need == (size_t)-1 ||
        (init && (init->scalar_type() != at::kFloat || init->sizes() != at::IntArrayRef(states))))
        Py_RETURN_NONE;
    at::Tensor y = make(x.t->sizes(), x.t->scalar_type(), *x.t);
    at::Tensor final_state = make(states, at::kFloat, *x.t), kept, ws = scratch(need, *x.t);
    if (keep) kept = make({(q.tokens + 63) / 64, width}, at::kFloat, *x.t);
    const ssd_status st = ssd_gated_scan_fwd(
        ptr(x.t), ptr(g.t), ptr(z.t), (ssd_dtype)c, q.nseq, q.length, q.offsets(), q.device,
        (int)width, x.stride, g.stride, z.stride, fptr(init), out(y), width, out<float>(final_state),
        out<float>(kept), out(ws), need, c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, tuple4(wrap(y), wrap(final_state), wrap(kept), Py_NewRef(Py_None)));
    END_HANDLE_TH_ERRORS
}

// dy, x, g, checkpoints, z, init_state, dfinal, offsets, device offsets
// -> (dx, dg, dz or None, dinit)
PyObject *gated_scan_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 9;
    const Matrix x = ok ? matrix(args[1], -1, ok) : Matrix();
    if (!ok || !x.t || x.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x.t->get_device();
    const Matrix dy = matrix(args[0], dev, ok), g = matrix(args[2], dev, ok);
    const Matrix z = matrix(args[4], dev, ok);
    const at::Tensor *kept = tensor(args[3], dev, ok), *init = tensor(args[5], dev, ok);
    const at::Tensor *dfinal = tensor(args[6], dev, ok);
    const int c = code(x.t->scalar_type());
    Sequences q;
    if (!ok || !dy.t || !g.t || !kept || !like(dy, *x.t) || !like(g, *x.t) || !like(z, *x.t) ||
        c < 0 || !sequences(*x.t, args[7], args[8], q))
        Py_RETURN_NONE;
    const int64_t width = x.t->size(-1);
    const std::array<int64_t, 2> states{q.nseq, width}, keeps{(q.tokens + 63) / 64, width};
    const auto is = [](const at::Tensor *t, at::IntArrayRef shape) {
        return !t || (t->scalar_type() == at::kFloat && t->sizes() == shape);
    };
    const size_t need = ssd_gated_scan_workspace_bytes((ssd_dtype)c, q.tokens, (int)width);
    if (need == (size_t)-1 || !is(init, states) || !is(dfinal, states) || !is(kept, keeps))
        Py_RETURN_NONE;
    const auto type = x.t->scalar_type();
    at::Tensor dx = make(x.t->sizes(), type, *x.t), dg = make(x.t->sizes(), type, *x.t), dz;
    if (z.t) dz = make(x.t->sizes(), type, *x.t);
    at::Tensor dinit = make(states, at::kFloat, *x.t), ws = scratch(need, *x.t);
    const ssd_status st = ssd_gated_scan_bwd(
        ptr(dy.t), ptr(x.t), ptr(g.t), ptr(z.t), (ssd_dtype)c, q.nseq, q.length, q.offsets(),
        q.device, (int)width, dy.stride, x.stride, g.stride, z.stride, fptr(init), fptr(kept),
        fptr(dfinal), out(dx), width, out(dg), width, out(dz), width, out<float>(dinit), out(ws),
        need, c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, tuple4(wrap(dx), wrap(dg), wrap(dz), wrap(dinit)));
    END_HANDLE_TH_ERRORS
}

#define SSD_METHOD(name) {#name, (PyCFunction)(void (*)())name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    SSD_METHOD(rmsnorm_fwd),
    SSD_METHOD(rmsnorm_bwd),
    SSD_METHOD(linear_fwd),
    SSD_METHOD(linear_bwd),
    SSD_METHOD(gated_scan_fwd),
    SSD_METHOD(gated_scan_bwd),
    SSD_METHOD(gated_state_update),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ssd_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ssd_marshal(void) { return PyModule_Create(&module); }
