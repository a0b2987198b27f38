// Argument marshalling of single-token calls: the same C entry points as the
// ctypes binding's (layer_ops.py), reached from tensors in one C call.  A call of
// one token lasts a few microseconds on the GPU and, through ctypes, 15 on the
// host: most of it Python's attribute and allocation calls.
//
// Each function answers plain calls (contiguous tensors of expected types and
// shapes on the current device, outputs to be allocated) and returns None for any
// other, which the Python code then takes: every refusal, message and layout is
// decided there.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

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
    const at::Tensor *x = ok ? tensor(args[1], -1, ok) : nullptr;
    if (!x || x->dim() < 2 || x->get_device() != c10::cuda::current_device()) Py_RETURN_NONE;
    const int dev = x->get_device();
    const at::Tensor *state = tensor(args[0], dev, ok), *g = tensor(args[2], dev, ok);
    const at::Tensor *z = tensor(args[3], dev, ok);
    if (!ok || !state || !g || state->scalar_type() != at::kFloat ||
        state->sizes() != x->sizes() || g->sizes() != x->sizes() ||
        g->scalar_type() != x->scalar_type() ||
        (z && (z->sizes() != x->sizes() || z->scalar_type() != x->scalar_type())))
        Py_RETURN_NONE;
    const int xc = code(x->scalar_type());
    if (xc < 0) Py_RETURN_NONE;
    const int64_t width = x->size(-1);
    at::Tensor y = make(x->sizes(), x->scalar_type(), *x);
    const ssd_status st = ssd_gated_state_update(
        state->mutable_data_ptr<float>(), ptr(x), ptr(g), ptr(z), (ssd_dtype)xc,
        x->numel() / width, (int)width, width, width, width, y.mutable_data_ptr(),
        c10::cuda::getCurrentCUDAStream(dev));
    return answer(st, THPVariable_Wrap(y));
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"rmsnorm_fwd", (PyCFunction)(void (*)())rmsnorm_fwd, METH_FASTCALL, nullptr},
    {"linear_fwd", (PyCFunction)(void (*)())linear_fwd, METH_FASTCALL, nullptr},
    {"gated_state_update", (PyCFunction)(void (*)())gated_state_update, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ssd_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ssd_marshal(void) { return PyModule_Create(&module); }
