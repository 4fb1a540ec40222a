// The binding's short way from tensors to the C ABI: the calls around the MX
// product take a few microseconds on the GPU, as long as checking eight tensors
// from Python does (a call from Python alone and this way: layer norm of one row
// 6.4 and 4.0 us, its gradient 512 x 512 9.2 and 4.4, quantize 512 x 512 5.3 and
// 4.0).
//
// Every function takes its Python namesake's tensors and scalars in order,
// workspace excluded, for tensors on torch's current device and its current
// stream.  It returns the C entry's code, or None, with nothing done, for
// arguments that are not exactly as the Python function wants them or on another
// device; that one then makes their device current or says what is wrong with them.
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include "tsgemm.h"

namespace {

// the library that the binding loaded
decltype(&tsgemm_layer_norm) p_layer_norm;
decltype(&tsgemm_layer_norm_grad_workspace) p_layer_norm_grad_workspace;
decltype(&tsgemm_layer_norm_grad) p_layer_norm_grad;
decltype(&tsgemm_mx_quantize) p_mx_quantize;
decltype(&tsgemm_mx_dequantize) p_mx_dequantize;
decltype(&tsgemm_mx_weight_grad_workspace) p_mx_weight_grad_workspace;
decltype(&tsgemm_mx_weight_grad) p_mx_weight_grad;
PyObject* raw_stream;             // device index -> handle of torch's current stream
int (*p_current_device)(int* dev);  // hipGetDevice of the runtime that the library launches with; NULL: one device only

int code_of(at::ScalarType t) {
    return t == at::kHalf ? TSGEMM_FP16 : t == at::kBFloat16 ? TSGEMM_BF16 : t == at::kFloat ? TSGEMM_FP32 : 0;
}

// The arguments of one call, read in order; `ok` falls when one is not as wanted.
struct Args {
    PyObject* const* at;
    bool ok = true;
    int dev = -1;
    int64_t rows = 0, width = 0;

    const at::Tensor* tensor(bool may_be_none = false) {
        PyObject* o = *at++;
        if (o == Py_None) {
            ok = ok && may_be_none;
            return nullptr;
        }
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor* t = &THPVariable_Unpack(o);
        if (!t->is_cuda() || t->layout() != at::kStrided) ok = false;
        else if (dev < 0) dev = t->get_device();
        else if (dev != t->get_device()) ok = false;
        return ok ? t : nullptr;
    }
    // a matrix with contiguous rows: its distance between rows
    int64_t row_stride(const at::Tensor& t) {
        const int64_t r = t.size(0), w = t.size(1), ld = r <= 1 ? w : t.stride(0);
        if ((t.stride(1) != 1 && w > 1) || ld < w) ok = false;
        return ld;
    }
    // the call's first matrix says how many rows and columns there are
    const at::Tensor* first(int64_t* ld) {
        const at::Tensor* t = tensor();
        if (!t) return nullptr;
        if (t->dim() != 2 || !code_of(t->scalar_type())) {
            ok = false;
            return nullptr;
        }
        rows = t->size(0);
        width = t->size(1);
        *ld = row_stride(*t);
        return t;
    }
    void* matrix(at::ScalarType type, int64_t* ld, bool may_be_none = false) {
        const at::Tensor* t = tensor(may_be_none);
        if (!t) return nullptr;
        if (t->dim() != 2 || t->size(0) != rows || t->size(1) != width || t->scalar_type() != type) {
            ok = false;
            return nullptr;
        }
        *ld = row_stride(*t);
        return t->data_ptr();
    }
    // a contiguous vector; an undefined `type` takes the first given one's
    void* vector(at::ScalarType* type, int64_t n, bool may_be_none) {
        const at::Tensor* t = tensor(may_be_none);
        if (!t) return nullptr;
        if (*type == at::ScalarType::Undefined) *type = t->scalar_type();
        if (t->dim() != 1 || t->size(0) != n || t->scalar_type() != *type || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void* bytes(int64_t columns, bool may_be_none) {
        const at::Tensor* t = tensor(may_be_none);
        if (!t) return nullptr;
        if (t->dim() != 2 || t->size(0) != rows || t->size(1) != columns || t->element_size() != 1 ||
            t->scalar_type() == at::kBool || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    // the stream to launch on, of the tensors' device, which has to be the current one
    void* stream() {
        int here = -1;
        if (p_current_device && (p_current_device(&here) != 0 || here != dev)) {
            ok = false;
            return nullptr;
        }
        PyObject* d = PyLong_FromLong(dev);
        PyObject* h = d ? PyObject_CallOneArg(raw_stream, d) : nullptr;
        Py_XDECREF(d);
        void* s = h ? PyLong_AsVoidPtr(h) : nullptr;
        Py_XDECREF(h);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return s;
    }
};

// A workspace of torch's allocator, taken for torch's current stream.
at::Tensor workspace(int64_t n, const at::Tensor& like) {
    return n > 0 ? at::empty({n}, like.options().dtype(at::kByte)) : at::Tensor();
}

template <class F>
PyObject* run(F&& call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// No C++ exception passes into Python: a call that threw has done nothing yet.
template <class F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "setup takes eight addresses and a function");
        return nullptr;
    }
    void* p[8];
    for (int i = 0; i < 8; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
    p_layer_norm = reinterpret_cast<decltype(p_layer_norm)>(p[0]);
    p_layer_norm_grad_workspace = reinterpret_cast<decltype(p_layer_norm_grad_workspace)>(p[1]);
    p_layer_norm_grad = reinterpret_cast<decltype(p_layer_norm_grad)>(p[2]);
    p_mx_quantize = reinterpret_cast<decltype(p_mx_quantize)>(p[3]);
    p_mx_dequantize = reinterpret_cast<decltype(p_mx_dequantize)>(p[4]);
    p_mx_weight_grad_workspace = reinterpret_cast<decltype(p_mx_weight_grad_workspace)>(p[5]);
    p_mx_weight_grad = reinterpret_cast<decltype(p_mx_weight_grad)>(p[6]);
    p_current_device = reinterpret_cast<decltype(p_current_device)>(p[7]);
    Py_INCREF(a[8]);
    Py_XSETREF(raw_stream, a[8]);
    Py_RETURN_NONE;
}

// x, gamma, beta, eps, y, mean, rstd, codes, scales
PyObject* layer_norm(PyObject*, PyObject* const* av, Py_ssize_t n) {
    if (n != 9) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a{av};
        int64_t ldx = 0, ldy = 0;
        const at::Tensor* x = a.first(&ldx);
        if (!a.ok) Py_RETURN_NONE;
        const at::ScalarType type = x->scalar_type();
        at::ScalarType wtype = at::ScalarType::Undefined, f32 = at::kFloat;
        const void* gamma = a.vector(&wtype, a.width, true);
        const void* beta = a.vector(&wtype, a.width, true);
        if (wtype == at::ScalarType::Undefined) wtype = type;
        const double eps = PyFloat_Check(*a.at) ? PyFloat_AS_DOUBLE(*a.at) : (a.ok = false, 0.0);
        ++a.at;
        void* y = a.matrix(type, &ldy, true);
        float* mean = static_cast<float*>(a.vector(&f32, a.rows, true));
        float* rstd = static_cast<float*>(a.vector(&f32, a.rows, true));
        void* codes = nullptr;
        void* scales = nullptr;
        if (av[7] != Py_None || av[8] != Py_None) {
            codes = a.bytes(a.width, false);
            scales = a.bytes(a.width / 32, false);
            a.ok = a.ok && a.width % 32 == 0;
        }
        void* s = a.ok ? a.stream() : nullptr;
        if (!a.ok || !code_of(wtype)) Py_RETURN_NONE;
        return run([&] {
            return p_layer_norm(a.rows, a.width, code_of(type), code_of(wtype), x->data_ptr(), ldx, gamma, beta,
                                static_cast<float>(eps), y, ldy, mean, rstd, codes, scales, s);
        });
    });
}

// dy, x, gamma, mean, rstd, dx, dgamma, dbeta
PyObject* layer_norm_grad(PyObject*, PyObject* const* av, Py_ssize_t n) {
    if (n != 8) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a{av};
        int64_t lddy = 0, ldx = 0, lddx = 0;
        const at::Tensor* dy = a.first(&lddy);
        if (!a.ok) Py_RETURN_NONE;
        const at::ScalarType type = dy->scalar_type();
        at::ScalarType wtype = at::ScalarType::Undefined, f32 = at::kFloat;
        const void* x = a.matrix(type, &ldx);
        const void* gamma = a.vector(&wtype, a.width, true);
        const float* mean = static_cast<const float*>(a.vector(&f32, a.rows, false));
        const float* rstd = static_cast<const float*>(a.vector(&f32, a.rows, false));
        void* dx = a.matrix(type, &lddx);
        void* dgamma = a.vector(&wtype, a.width, true);
        void* dbeta = a.vector(&wtype, a.width, true);
        if (wtype == at::ScalarType::Undefined) wtype = type;
        if (!a.ok || !code_of(wtype)) Py_RETURN_NONE;
        const int64_t need = dgamma || dbeta ? p_layer_norm_grad_workspace(a.rows, a.width) : 0;
        if (need < 0) Py_RETURN_NONE;
        void* s = a.stream();
        if (!a.ok) Py_RETURN_NONE;
        const at::Tensor ws = workspace(need, *dy);
        return run([&] {
            return p_layer_norm_grad(a.rows, a.width, code_of(type), code_of(wtype), dy->data_ptr(), lddy, x, ldx, gamma,
                                     mean, rstd, dx, lddx, dgamma, dbeta, need ? ws.data_ptr() : nullptr, need, s);
        });
    });
}

// x, codes, scales
PyObject* mx_quantize(PyObject*, PyObject* const* av, Py_ssize_t n) {
    if (n != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a{av};
        int64_t ld = 0;
        const at::Tensor* x = a.first(&ld);
        if (!a.ok || a.width % 32 != 0) Py_RETURN_NONE;
        void* codes = a.bytes(a.width, false);
        void* scales = a.bytes(a.width / 32, false);
        void* s = a.ok ? a.stream() : nullptr;
        if (!a.ok) Py_RETURN_NONE;
        return run([&] { return p_mx_quantize(a.rows, a.width, code_of(x->scalar_type()), x->data_ptr(), ld, codes, scales, s); });
    });
}

// out, codes, scales (the matrix first: it says how large the others are)
PyObject* mx_dequantize(PyObject*, PyObject* const* av, Py_ssize_t n) {
    if (n != 3) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a{av};
        int64_t ld = 0;
        const at::Tensor* out = a.first(&ld);
        if (!a.ok || a.width % 32 != 0) Py_RETURN_NONE;
        const void* codes = a.bytes(a.width, false);
        const void* scales = a.bytes(a.width / 32, false);
        void* s = a.ok ? a.stream() : nullptr;
        if (!a.ok) Py_RETURN_NONE;
        return run([&] { return p_mx_dequantize(a.rows, a.width, code_of(out->scalar_type()), codes, scales, out->data_ptr(), ld, s); });
    });
}

// dy, codes, scales, dw
PyObject* mx_weight_grad(PyObject*, PyObject* const* av, Py_ssize_t n) {
    if (n != 4) Py_RETURN_NONE;
    return guarded([&]() -> PyObject* {
        Args a{av};
        int64_t lddy = 0;
        const at::Tensor* dy = a.first(&lddy);
        if (!a.ok) Py_RETURN_NONE;
        const int64_t out = a.width;
        a.at = av + 3;
        const at::Tensor* dw = a.tensor();
        if (!a.ok || dw->dim() != 2 || dw->size(0) != out || !dw->is_contiguous() || !code_of(dw->scalar_type())) Py_RETURN_NONE;
        const int64_t width = dw->size(1);
        if (width % 32 != 0) Py_RETURN_NONE;
        a.at = av + 1;
        const void* codes = a.bytes(width, false);
        const void* scales = a.bytes(width / 32, false);
        if (!a.ok) Py_RETURN_NONE;
        const int64_t need = p_mx_weight_grad_workspace(a.rows, out, width);
        if (need < 0) Py_RETURN_NONE;
        void* s = a.stream();
        if (!a.ok) Py_RETURN_NONE;
        const at::Tensor ws = workspace(need, *dy);
        return run([&] {
            return p_mx_weight_grad(a.rows, out, width, code_of(dy->scalar_type()), code_of(dw->scalar_type()), dy->data_ptr(), lddy,
                                    codes, scales, dw->data_ptr(), need ? ws.data_ptr() : nullptr, need, s);
        });
    });
}

#define TSG_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TSG_METHOD(setup), TSG_METHOD(layer_norm), TSG_METHOD(layer_norm_grad), TSG_METHOD(mx_quantize),
                         TSG_METHOD(mx_dequantize), TSG_METHOD(mx_weight_grad), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tsgemm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tsgemm_torch() { return PyModule_Create(&module); }
