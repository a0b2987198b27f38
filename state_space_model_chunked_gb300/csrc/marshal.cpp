// Argument marshalling of small calls: the same C entry points as the ctypes
// binding's (layer_ops.py), reached from tensors in one C call.  A call of one
// token lasts a few microseconds on the GPU and, through ctypes, 15 on the host:
// most of it Python's attribute and allocation calls.
//
// Each function answers plain calls (tensors of expected types and shapes on the
// current device, outputs and workspace to be allocated) and returns None for any
// other, which the Python code then takes: every refusal, message and further
// layout is decided there.
#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <climits>
#include <cmath>

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

// A new array.  Past torch's dispatcher, which takes half a microsecond of the host's time
// (a layer norm of a few tokens makes four: 10.1 -> 7.9 us a call), unless it has to fill the
// array, or a dispatch mode (or another layer that is on in this thread) is to see it.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like) {
    if (at::globalContext().deterministicAlgorithms() ||
        c10::impl::tls_local_dispatch_key_set().included_ != c10::default_included_set)
        return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
    return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
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

// The sequences of a recurrence over tokens [batch, length], or [tokens] with offsets as a
// list of ints and their device copy.
struct Sequences {
    int nseq = 0, length = 0;
    int64_t tokens = 0;
    c10::SmallVector<int, 64> host;
    const int *device = nullptr;
    const int *offsets() const { return host.empty() ? nullptr : host.data(); }
};
bool sequences(at::IntArrayRef lead, int device, PyObject *cu, PyObject *cu_dev, Sequences &s) {
    s.tokens = c10::multiply_integers(lead);
    if (s.tokens > INT_MAX) return false;
    if (cu == Py_None) {
        if (lead.size() != 2) return false;
        s.nseq = (int)lead[0];
        s.length = (int)lead[1];
        return true;
    }
    bool ok = lead.size() == 1 && PyList_Check(cu) && PyList_GET_SIZE(cu) >= 2;
    const at::Tensor *d = ok ? tensor(cu_dev, device, ok) : nullptr;
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
        !sequences(x.t->sizes().slice(0, x.t->dim() - 1), dev, args[4], args[5], q))
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
        c < 0 || !sequences(x.t->sizes().slice(0, x.t->dim() - 1), dev, args[7], args[8], q))
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

// A tuple of five.
PyObject *tuple5(PyObject *a, PyObject *b, PyObject *c, PyObject *d, PyObject *e) {
    PyObject *t = PyTuple_New(5);
    PyTuple_SET_ITEM(t, 0, a);
    PyTuple_SET_ITEM(t, 1, b);
    PyTuple_SET_ITEM(t, 2, c);
    PyTuple_SET_ITEM(t, 3, d);
    PyTuple_SET_ITEM(t, 4, e);
    return t;
}

// x, weight, bias or None, residual or None, eps, out code
// -> (y, residual_out or None, mean, rstd, scale or None)
PyObject *layernorm_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 6;
    const Matrix x = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !x.t || x.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x.t->get_device();
    const at::Tensor *w = tensor(args[1], dev, ok), *b = tensor(args[2], dev, ok);
    const Matrix r = matrix(args[3], dev, ok);
    const double eps = PyFloat_AsDouble(args[4]);
    const int out_code = (int)PyLong_AsLong(args[5]), xc = code(x.t->scalar_type());
    const int64_t width = x.t->size(-1), rows = x.t->numel() / width;
    if (PyErr_Occurred()) return nullptr;
    if (!ok || !w || !vector(w, width) || !vector(b, width) || xc < 0 ||
        (r.t && r.t->sizes() != x.t->sizes()))
        Py_RETURN_NONE;
    const int rc = r.t ? code(r.t->scalar_type()) : xc;
    if (rc < 0) Py_RETURN_NONE;
    const auto lead = x.t->sizes().slice(0, x.t->dim() - 1);
    at::Tensor y = make(x.t->sizes(), type_of(out_code), *x.t), mean = make(lead, at::kFloat, *x.t);
    at::Tensor rstd = make(lead, at::kFloat, *x.t), so, scale;
    if (r.t) so = make(x.t->sizes(), r.t->scalar_type(), *x.t);
    if (out_code == SSD_FP8_E4M3) scale = make(lead, at::kFloat, *x.t);
    const ssd_status st = ssd_layernorm_fwd(
        ptr(x.t), ptr(r.t), fptr(w), fptr(b), (float)eps, (ssd_dtype)xc, (ssd_dtype)rc,
        (ssd_dtype)out_code, rows, (int)width, x.stride, r.stride, out(y), out(so), out<float>(mean),
        out<float>(rstd), out<float>(scale), c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, tuple5(wrap(y), wrap(so), wrap(mean), wrap(rstd), wrap(scale)));
    END_HANDLE_TH_ERRORS
}

// dy, s, weight, mean, rstd, dresidual, whether dbias is wanted
// -> (dx, ds (dx itself for one type), dweight, dbias or None)
PyObject *layernorm_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 7;
    const Matrix dy = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !dy.t || dy.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = dy.t->get_device();
    const Matrix s = matrix(args[1], dev, ok), dr = matrix(args[5], dev, ok);
    const at::Tensor *w = tensor(args[2], dev, ok), *mean = tensor(args[3], dev, ok);
    const at::Tensor *rstd = tensor(args[4], dev, ok);
    const int bias = PyObject_IsTrue(args[6]);
    if (bias < 0) return nullptr;       // no truth value: the exception is set
    const int64_t width = dy.t->size(-1), rows = dy.t->numel() / width;
    const auto lead = dy.t->sizes().slice(0, dy.t->dim() - 1);
    const auto stat = [&](const at::Tensor *t) { return t && t->scalar_type() == at::kFloat && t->sizes() == lead; };
    if (!ok || !s.t || !w || s.t->sizes() != dy.t->sizes() || !like(dr, *s.t) || !vector(w, width) ||
        !stat(mean) || !stat(rstd))
        Py_RETURN_NONE;
    const int c = code(dy.t->scalar_type()), sc = code(s.t->scalar_type());
    const size_t need = ssd_layernorm_bwd_workspace_bytes(rows, (int)width);
    if (c < 0 || sc < 0 || need == (size_t)-1) Py_RETURN_NONE;
    at::Tensor dx = make(dy.t->sizes(), dy.t->scalar_type(), *dy.t), ds, db;
    if (c != sc) ds = make(dy.t->sizes(), s.t->scalar_type(), *dy.t);
    at::Tensor dw = make({width}, at::kFloat, *dy.t), ws = scratch(need, *dy.t);
    if (bias) db = make({width}, at::kFloat, *dy.t);
    const ssd_status st = ssd_layernorm_bwd(
        ptr(dy.t), ptr(s.t), fptr(w), fptr(mean), fptr(rstd), ptr(dr.t), (ssd_dtype)c, (ssd_dtype)sc,
        rows, (int)width, dy.stride, s.stride, dr.stride, out(dx), out(ds), out<float>(dw),
        out<float>(db), out(ws), need, c10::cuda::getCurrentCUDAStream(dev));
    PyObject *first = wrap(dx);
    return answer(st, tuple4(first, ds.defined() ? wrap(ds) : Py_NewRef(first), wrap(dw), wrap(db)));
    END_HANDLE_TH_ERRORS
}

// Token numbers: -1 for other types.
int index_code(const at::Tensor &t) {
    return t.scalar_type() == at::kInt ? SSD_I32 : (t.scalar_type() == at::kLong ? SSD_I64 : -1);
}

// tokens, table, scale, out code -> y
PyObject *embedding_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 4;
    const at::Tensor *ids = ok ? tensor(args[0], -1, ok) : nullptr;
    if (!ids || ids->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = ids->get_device();
    const at::Tensor *table = tensor(args[1], dev, ok);
    const double scale = PyFloat_AsDouble(args[2]);
    const int out_code = (int)PyLong_AsLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    if (!ok || !table || table->dim() != 2 || index_code(*ids) < 0 || code(table->scalar_type()) < 0)
        Py_RETURN_NONE;
    c10::SmallVector<int64_t, 6> shape(ids->sizes().begin(), ids->sizes().end());
    shape.push_back(table->size(1));
    at::Tensor y = make(shape, type_of(out_code), *table);
    const ssd_status st = ssd_embedding_fwd(
        ptr(ids), (ssd_index)index_code(*ids), ptr(table), (ssd_dtype)code(table->scalar_type()),
        (ssd_dtype)out_code, ids->numel(), (int)table->size(0), (int)table->size(1), (float)scale,
        out(y), c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, wrap(y));
    END_HANDLE_TH_ERRORS
}

// dy, tokens, vocab, scale, out code -> dtable
PyObject *embedding_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 5;
    const Matrix dy = ok ? matrix(args[0], -1, ok) : Matrix();
    if (!ok || !dy.t || dy.t->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = dy.t->get_device();
    const at::Tensor *ids = tensor(args[1], dev, ok);
    const long long vocab = PyLong_AsLongLong(args[2]);
    const double scale = PyFloat_AsDouble(args[3]);
    const int out_code = (int)PyLong_AsLong(args[4]);
    if (PyErr_Occurred()) return nullptr;
    const int64_t width = dy.t->size(-1);
    if (!ok || !ids || index_code(*ids) < 0 || code(dy.t->scalar_type()) < 0 || vocab <= 0 ||
        vocab > INT_MAX || ids->sizes() != dy.t->sizes().slice(0, dy.t->dim() - 1))
        Py_RETURN_NONE;
    const size_t need = ssd_embedding_bwd_workspace_bytes(ids->numel(), (int)vocab, (int)width);
    if (need == (size_t)-1) Py_RETURN_NONE;
    at::Tensor dtable = make({(int64_t)vocab, width}, type_of(out_code), *dy.t), ws = scratch(need, *dy.t);
    const ssd_status st = ssd_embedding_bwd(
        ptr(dy.t), ptr(ids), (ssd_index)index_code(*ids), (ssd_dtype)code(dy.t->scalar_type()),
        (ssd_dtype)out_code, ids->numel(), (int)vocab, (int)width, dy.stride, (float)scale, out(dtable),
        out(ws), need, c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, wrap(dtable));
    END_HANDLE_TH_ERRORS
}

// An array of a token's values a row: [..., a, b] with the last two dimensions contiguous
// and the rows at one stride (never None).
Matrix by_token(PyObject *o, int device, bool &ok) {
    Matrix m;
    if (!THPVariable_Check(o)) {
        ok = false;
        return m;
    }
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() < 3 || t.numel() == 0 || t.size(0) > INT_MAX || t.size(-2) > INT_MAX ||
        t.size(-1) > INT_MAX || (device >= 0 && t.get_device() != device) ||
        (t.size(-1) > 1 && t.stride(-1) != 1) || (t.size(-2) > 1 && t.stride(-2) != t.size(-1))) {
        ok = false;
        return m;
    }
    int64_t row = -1, step = 0;
    for (int64_t d = t.dim() - 3; d >= 0; --d) {
        if (t.size(d) == 1) continue;
        if (row < 0) row = t.stride(d);
        else if (t.stride(d) != step) ok = false;
        step = t.stride(d) * t.size(d);
    }
    m.t = &t;
    m.stride = row < 0 ? t.size(-2) * t.size(-1) : row;
    return m;
}

// What the passes over sequences of the delta rule have in common: q, k, v, g, beta, init or
// final state's gradient, scale or None, offsets, device offsets.
struct DeltaInputs {
    Matrix q, k, v;
    const at::Tensor *g = nullptr, *beta = nullptr, *state = nullptr;
    Sequences s;
    int dev = 0, code = -1, heads = 0, p = 0, n = 0, groups = 0;
    float scale = 0;
    std::array<int64_t, 4> states{}, kept{};
};
// Whether they are such; false with an exception set where Python raised one.
bool delta_inputs(PyObject *const *args, PyObject *scale, PyObject *cu, PyObject *cu_dev, DeltaInputs &d) {
    bool ok = true;
    d.q = by_token(args[0], -1, ok);
    if (!ok || d.q.t->get_device() != c10::cuda::current_device()) return false;
    const at::Tensor &q = *d.q.t;
    d.dev = q.get_device();
    d.k = by_token(args[1], d.dev, ok);
    d.v = by_token(args[2], d.dev, ok);
    d.g = tensor(args[3], d.dev, ok);
    d.beta = tensor(args[4], d.dev, ok);
    d.state = tensor(args[5], d.dev, ok);
    if (!ok || !d.g || !d.beta) return false;
    const at::Tensor &v = *d.v.t;
    const auto lead = q.sizes().slice(0, q.dim() - 2);
    const auto gate = [&](const at::Tensor *t) {
        return t->scalar_type() == at::kFloat && t->sizes() == v.sizes().slice(0, v.dim() - 1);
    };
    if (!like(d.k, q) || v.scalar_type() != q.scalar_type() || v.sizes().slice(0, v.dim() - 2) != lead ||
        !gate(d.g) || !gate(d.beta) || !sequences(lead, d.dev, cu, cu_dev, d.s))
        return false;
    d.code = code(q.scalar_type());
    d.groups = (int)q.size(-2);
    d.n = (int)q.size(-1);
    d.heads = (int)v.size(-2);
    d.p = (int)v.size(-1);
    d.scale = (float)(scale == Py_None ? std::pow((double)d.n, -0.5) : PyFloat_AsDouble(scale));
    if (PyErr_Occurred()) return false;
    d.states = {d.s.nseq, d.heads, d.p, d.n};
    d.kept = {d.s.tokens / 64 + d.s.nseq, d.heads, d.p, d.n};
    return d.code >= 0 && (!d.state || (d.state->scalar_type() == at::kFloat && d.state->sizes() == at::IntArrayRef(d.states)));
}

// q, k, v, g, beta, init_state, scale or None, offsets, device offsets, whether the final
// state and the checkpoints are wanted -> (o, final_state or None, checkpoints or None, None)
PyObject *delta_scan_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    DeltaInputs d;
    if (n != 11 || !delta_inputs(args, args[6], args[7], args[8], d)) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
    const int last = PyObject_IsTrue(args[9]), keep = last < 0 ? -1 : PyObject_IsTrue(args[10]);
    if (keep < 0) return nullptr;       // no truth value: the exception is set
    const size_t need = ssd_delta_scan_workspace_bytes((ssd_dtype)d.code, d.s.tokens, d.s.nseq, d.heads, d.p, d.n, d.groups);
    if (need == (size_t)-1) Py_RETURN_NONE;
    const at::Tensor &q = *d.q.t;
    at::Tensor o = make(d.v.t->sizes(), q.scalar_type(), q), final_state, kept, ws = scratch(need, q);
    if (last) final_state = make(d.states, at::kFloat, q);
    if (keep) kept = make(d.kept, at::kFloat, q);
    const ssd_status st = ssd_delta_scan_fwd(
        ptr(d.q.t), ptr(d.k.t), ptr(d.v.t), fptr(d.g), fptr(d.beta), (ssd_dtype)d.code, d.s.nseq, d.s.length,
        d.s.offsets(), d.s.device, d.heads, d.p, d.n, d.groups, d.q.stride, d.k.stride, d.v.stride, d.scale,
        fptr(d.state), out(o), (int64_t)d.heads * d.p, out<float>(final_state), out<float>(kept), out(ws), need,
        c10::cuda::getCurrentCUDAStream(d.dev));
    return answer(st, tuple4(wrap(o), wrap(final_state), wrap(kept), Py_NewRef(Py_None)));
    END_HANDLE_TH_ERRORS
}

// q, k, v, g, beta, dfinal, do, checkpoints, scale or None, offsets, device offsets, whether
// dinit is wanted -> (dq, dk, dv, dg, dbeta, dinit or None)
PyObject *delta_scan_bwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    DeltaInputs d;
    if (n != 12 || !delta_inputs(args, args[8], args[9], args[10], d)) {
        if (PyErr_Occurred()) return nullptr;
        Py_RETURN_NONE;
    }
    bool ok = true;
    const Matrix dout = by_token(args[6], d.dev, ok);
    const at::Tensor *kept = tensor(args[7], d.dev, ok);
    const int init = PyObject_IsTrue(args[11]);
    if (init < 0) return nullptr;       // no truth value: the exception is set
    const at::Tensor &q = *d.q.t, &v = *d.v.t;
    if (!ok || !like(dout, v) || !kept || kept->scalar_type() != at::kFloat || kept->sizes() != at::IntArrayRef(d.kept))
        Py_RETURN_NONE;
    // the workspace of the kernels that run: where everything lies on 16 bytes the tensor cores'
    // (0: not for these sizes), else the others'
    uintptr_t where = (uintptr_t)((dout.stride | d.q.stride | d.k.stride | d.v.stride) * q.element_size());
    for (const at::Tensor *t : {dout.t, d.q.t, d.k.t, d.v.t, kept, d.state}) where |= (uintptr_t)ptr(t);
    const auto size = [&](ssd_algo algo) {
        return ssd_delta_scan_bwd_workspace_bytes_algo(algo, (ssd_dtype)d.code, d.s.tokens, d.s.nseq, d.heads, d.p, d.n, d.groups);
    };
    size_t need = where % 16 == 0 ? size(SSD_ALGO_TCGEN05) : 0;
    if (need == 0) need = size(SSD_ALGO_SIMT);
    if (need == (size_t)-1) Py_RETURN_NONE;
    const auto type = q.scalar_type();
    at::Tensor dq = make(q.sizes(), type, q), dk = make(q.sizes(), type, q), dv = make(v.sizes(), type, q);
    at::Tensor dg = make(d.g->sizes(), at::kFloat, q), dbeta = make(d.g->sizes(), at::kFloat, q), dinit;
    if (init) dinit = make(d.states, at::kFloat, q);
    at::Tensor ws = scratch(need, q);
    const int64_t keys = (int64_t)d.groups * d.n, values = (int64_t)d.heads * d.p;
    const ssd_status st = ssd_delta_scan_bwd(
        ptr(dout.t), ptr(d.q.t), ptr(d.k.t), ptr(d.v.t), fptr(d.g), fptr(d.beta), (ssd_dtype)d.code, d.s.nseq,
        d.s.length, d.s.offsets(), d.s.device, d.heads, d.p, d.n, d.groups, dout.stride, d.q.stride, d.k.stride,
        d.v.stride, d.scale, fptr(kept), fptr(d.state), out(dq), keys, out(dk), keys, out(dv), values,
        out<float>(dg), out<float>(dbeta), out<float>(dinit), out(ws), need, c10::cuda::getCurrentCUDAStream(d.dev));
    PyObject *t = PyTuple_New(6);
    int at = 0;
    for (const at::Tensor *x : {&dq, &dk, &dv, &dg, &dbeta, &dinit}) PyTuple_SET_ITEM(t, at++, wrap(*x));
    return answer(st, t);
    END_HANDLE_TH_ERRORS
}

// state, q, k, v, g, beta, scale or None, state_out or None -> o
PyObject *delta_state_update(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    bool ok = n == 8;
    const at::Tensor *state = ok ? tensor(args[0], -1, ok) : nullptr;
    if (!state || state->dim() != 4 || state->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = state->get_device();
    const Matrix q = by_token(args[1], dev, ok), k = by_token(args[2], dev, ok), v = by_token(args[3], dev, ok);
    const at::Tensor *g = tensor(args[4], dev, ok), *beta = tensor(args[5], dev, ok);
    const at::Tensor *next = tensor(args[7], dev, ok);
    if (!ok || !g || !beta) Py_RETURN_NONE;
    const int64_t batch = state->size(0), heads = state->size(1), p = state->size(2), s = state->size(3);
    const double scale = args[6] == Py_None ? std::pow((double)s, -0.5) : PyFloat_AsDouble(args[6]);
    if (PyErr_Occurred()) return nullptr;
    const std::array<int64_t, 2> gates{batch, heads};
    const std::array<int64_t, 3> values{batch, heads, p}, keys{batch, q.t->size(1), s};
    const auto gate = [&](const at::Tensor *t) {
        return t->scalar_type() == at::kFloat && t->sizes() == at::IntArrayRef(gates);
    };
    if (heads > INT_MAX || p > INT_MAX || v.t->sizes() != at::IntArrayRef(values) ||
        q.t->sizes() != at::IntArrayRef(keys) || !like(k, *q.t) || v.t->scalar_type() != q.t->scalar_type() ||
        !gate(g) || !gate(beta) || code(q.t->scalar_type()) < 0 || code(state->scalar_type()) < 0 ||
        (next && (next->sizes() != state->sizes() || next->scalar_type() != state->scalar_type())))
        Py_RETURN_NONE;
    at::Tensor o = make(values, q.t->scalar_type(), *q.t);
    const ssd_status st = ssd_delta_state_update(
        ptr(state), (ssd_dtype)code(state->scalar_type()), (next ? next : state)->mutable_data_ptr(),
        ptr(q.t), ptr(k.t), ptr(v.t), fptr(g), fptr(beta), (ssd_dtype)code(q.t->scalar_type()), (int)batch,
        (int)heads, (int)p, (int)s, (int)q.t->size(1), q.stride, k.stride, v.stride, (float)scale, out(o),
        c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, wrap(o));
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
    SSD_METHOD(layernorm_fwd),
    SSD_METHOD(layernorm_bwd),
    SSD_METHOD(embedding_fwd),
    SSD_METHOD(embedding_bwd),
    SSD_METHOD(delta_state_update),
    SSD_METHOD(delta_scan_fwd),
    SSD_METHOD(delta_scan_bwd),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ssd_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ssd_marshal(void) { return PyModule_Create(&module); }
