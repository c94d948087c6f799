// dwc_norm_py.cpp -- host path of the norm and dropout operators for Python (CPython C API).
//
// Small calls are bound by the host: through ctypes and tensor attributes read one by one a
// backward pass cost 23 us of Python beside 13 us of GPU work.  Here the checks, the outputs'
// allocation (PyTorch's allocator, so memory belongs to the current stream or graph) and the
// call of the C ABI (include/dwc_norm.h) are one C++ function per operator.  Nothing is computed
// here and nothing is kept between calls.  norm.py documents the functions and handles `stream`.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>

#include "../../include/dwc_norm.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;   // DwcError(function, code), given by norm.py

struct Failed {                // a status code of the library
    const char* fn;
    int code;
};

dwc_dtype_t code_of(ScalarType t) {
    switch (t) {
        case ScalarType::Float: return DWC_F32;
        case ScalarType::BFloat16: return DWC_BF16;
        case ScalarType::Half: return DWC_F16;
        default: TORCH_CHECK_TYPE(false, "unsupported dtype ", t, " (fp32, bf16 or fp16)");
    }
}

const Tensor& tensor(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
    return THPVariable_Unpack(o);
}

// Elements between the rows of [..., C]: one stride over all leading axes, adjacent channels.
int64_t row_stride(const Tensor& t, const char* what) {
    const auto shape = t.sizes(), stride = t.strides();
    const int64_t C = shape.back();
    if (t.is_contiguous()) return C;
    TORCH_CHECK_VALUE(C == 1 || stride.back() == 1, what, ": channels must be adjacent (stride ", stride.back(), ")");
    int64_t ld = -1, span = 0;
    for (int64_t i = t.dim() - 2; i >= 0; --i) {
        if (shape[i] == 1) continue;
        if (ld < 0) {
            TORCH_CHECK_VALUE(stride[i] >= C, what, ": rows overlap (stride ", stride[i], " between rows of ", C, ")");
            ld = stride[i];
            span = ld * shape[i];
        } else {
            TORCH_CHECK_VALUE(stride[i] == span, what, ": rows must have one stride (got ", stride, " for ", shape, ")");
            span *= shape[i];
        }
    }
    return ld < 0 ? C : ld;
}

// A new dense tensor from PyTorch's allocator (the CUDA backend's own factory: the dispatcher's way
// to it costs as much again).
Tensor new_tensor(at::IntArrayRef shape, ScalarType type, const at::Device& device) {
    return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// The tensor whose shape, device and channels a call goes by.
struct Rows {
    const Tensor& t;
    int64_t C, rows, ld;
    Rows(const Tensor& x, const char* what) : t(x) {
        TORCH_CHECK_VALUE(x.is_cuda(), "tensors must be on a CUDA device (no CPU fallback)");
        TORCH_CHECK_VALUE(x.dim() >= 1 && x.size(-1) >= 1, what, " must be [..., C] with at least one channel");
        C = x.size(-1);
        TORCH_CHECK_VALUE(C <= INT32_MAX, what, " has more channels than the library takes");
        rows = x.numel() / C;
        ld = row_stride(x, what);
    }
    int64_t like(const Tensor& o, const char* what) const {
        TORCH_CHECK_VALUE(o.sizes() == t.sizes() && o.device() == t.device(), what, " must be a ", t.sizes(),
                          " tensor on ", t.device(), " (got ", o.sizes(), " on ", o.device(), ")");
        return row_stride(o, what);
    }
    // a dense output: the caller's, checked, or a new one
    Tensor out(PyObject* o, ScalarType type, const char* what) const {
        if (o == Py_None) return new_tensor(t.sizes(), type, t.device());
        const Tensor& given = tensor(o, what);
        TORCH_CHECK_VALUE(given.sizes() == t.sizes() && given.scalar_type() == type && given.device() == t.device() &&
                              given.is_contiguous(),
                          what, " must be a contiguous ", t.sizes(), " ", type, " tensor on ", t.device(), " (got ",
                          given.sizes(), " ", given.scalar_type(), " on ", given.device(), ")");
        return given;
    }
    Tensor stat() const {
        return new_tensor(t.sizes().slice(0, t.dim() - 1), at::kFloat, t.device());
    }
    const float* given_stat(PyObject* o, const char* what) const {
        const Tensor& s = tensor(o, what);
        const auto lead = t.sizes().slice(0, t.dim() - 1);
        TORCH_CHECK_VALUE(s.sizes() == lead && s.scalar_type() == at::kFloat && s.device() == t.device() && s.is_contiguous(),
                          what, " must be a contiguous ", lead, " fp32 tensor on ", t.device(), " (got ", s.sizes(), " ",
                          s.scalar_type(), " on ", s.device(), ")");
        return static_cast<const float*>(s.data_ptr());
    }
};

// An output given by the caller may be one of the call's inputs, from the same address, dense and of its type
// (an update in place); it must not overlap inputs or another output in any other way.  `in`: rows of
// C elements, ld apart.
void check_apart(const Tensor& out, const char* what, const Tensor& in, int64_t rows, int64_t C, int64_t ld,
                 const char* name, bool may_be = true) {
    const auto o = reinterpret_cast<uintptr_t>(out.data_ptr()), b = reinterpret_cast<uintptr_t>(in.data_ptr());
    const uintptr_t end = o + out.numel() * out.element_size(), size = in.element_size(), width = C * size, step = ld * size;
    if (o == end || rows == 0 || end <= b || o >= b + (rows - 1) * step + width) return;
    if (may_be && o == b && out.scalar_type() == in.scalar_type() && out.sizes() == in.sizes() && in.is_contiguous()) return;
    // the first row that ends past the output's start
    const uintptr_t row = o < b + width ? 0 : (o - b - width) / step + 1;
    TORCH_CHECK_VALUE(b + row * step >= end, what, " overlaps ", name,
                      may_be ? " (it may be a dense tensor of its dtype itself, but not a part of it)" : "");
}
void check_apart(const Tensor& out, const char* what, PyObject* vector, const char* name) {
    if (!THPVariable_Check(vector)) return;
    const Tensor& t = THPVariable_Unpack(vector);
    if (t.numel() > 0) check_apart(out, what, t, 1, t.numel(), t.numel(), name, false);
}

// gamma and beta: C values of one type each, or None.
struct Params {
    const void* p[2] = {nullptr, nullptr};
    dwc_dtype_t type = DWC_F32;
    Params(const Rows& x, PyObject* gamma, PyObject* beta) {
        bool any = false;
        for (int i = 0; i < 2; ++i) {
            PyObject* o = i == 0 ? gamma : beta;
            if (o == Py_None) continue;
            const Tensor& t = tensor(o, i == 0 ? "gamma" : "beta");
            TORCH_CHECK_VALUE(t.dim() == 1 && t.numel() == x.C && t.device() == x.t.device() && t.is_contiguous(),
                              i == 0 ? "gamma" : "beta", " must hold ", x.C, " values on ", x.t.device(), " (got ",
                              t.sizes(), " on ", t.device(), ")");
            const dwc_dtype_t c = code_of(t.scalar_type());
            TORCH_CHECK_VALUE(!any || c == type, "gamma and beta must have one dtype");
            type = c;
            any = true;
            p[i] = t.data_ptr();
        }
    }
};

unsigned long long word64(PyObject* o) {
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (PyErr_Occurred()) throw python_error();
    return v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

// p, seed and offset of a dropout; an offset may be one int64 value on the device.
struct Random {
    double p;
    unsigned long long seed, offset = 0;
    const unsigned long long* step = nullptr;
    Random(const Rows& x, PyObject* prob, PyObject* seed_, PyObject* offset_) : p(number(prob)), seed(word64(seed_)) {
        TORCH_CHECK_VALUE(p >= 0.0 && p <= 1.0, "p must be in [0, 1] (got ", p, ")");
        if (!THPVariable_Check(offset_)) {
            offset = word64(offset_);
            return;
        }
        const Tensor& t = THPVariable_Unpack(offset_);
        TORCH_CHECK_VALUE(t.scalar_type() == at::kLong && t.numel() == 1 && t.device() == x.t.device(),
                          "an offset on the device must be one int64 value on the tensors' device");
        step = static_cast<const unsigned long long*>(t.data_ptr());
    }
};

// The current stream of the tensors' device, with that device current.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    dwc_stream_t stream;
    explicit OnDevice(const Rows& x) {
        const auto index = x.t.get_device();
        if (index != c10::cuda::current_device()) guard.set_index(index);
        stream = c10::cuda::getCurrentCUDAStream(index).stream();
    }
};

void check(const char* fn, dwc_status_t code) {
    if (code != DWC_OK) throw Failed{fn, static_cast<int>(code)};
}

// dgamma, dbeta and the workspace of a backward pass.
struct ParamGrads {
    Tensor dgamma, dbeta, ws;
    float *dg = nullptr, *db = nullptr;
    void* w = nullptr;
    size_t bytes = 0;
    ParamGrads(const Rows& x, bool wanted) {
        if (!wanted) return;
        dgamma = new_tensor({x.C}, at::kFloat, x.t.device());
        dbeta = new_tensor({x.C}, at::kFloat, x.t.device());
        bytes = dwc_layer_norm_bwd_workspace_size(x.rows, static_cast<int>(x.C));
        ws = new_tensor({static_cast<int64_t>(bytes)}, at::kByte, x.t.device());
        dg = static_cast<float*>(dgamma.data_ptr());
        db = static_cast<float*>(dbeta.data_ptr());
        w = ws.data_ptr();
    }
};

PyObject* wrap(const Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject* pack(std::initializer_list<const Tensor*> list) {
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(list.size()));
    if (tuple == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor* t : list) {
        PyObject* o = wrap(*t);
        if (o == nullptr) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

float* fp(const Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }

using Fast = PyObject* (*)(PyObject* const*);

// The common frame: the number of arguments, and every C++ exception as a Python one.
template <Fast f, int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    TORCH_CHECK_TYPE(n == kArgs, "expected ", kArgs, " arguments, got ", n);
    try {
        return f(a);
    } catch (const Failed& e) {
        if (PyObject* x = PyObject_CallFunction(g_error, "si", e.fn, e.code)) {
            PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(x)), x);
            Py_DECREF(x);
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (x, gamma, beta, eps, out, out_dtype, stats)
PyObject* layer_norm_fwd(PyObject* const* a) {
    const Rows x(tensor(a[0], "x"), "x");
    const Params w(x, a[1], a[2]);
    ScalarType type = x.t.scalar_type();
    if (a[5] != Py_None) {
        TORCH_CHECK_TYPE(THPDtype_Check(a[5]), "out_dtype must be a dtype");
        type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    } else if (a[4] != Py_None) {
        type = tensor(a[4], "out").scalar_type();
    }
    const dwc_dtype_t in = code_of(x.t.scalar_type()), od = code_of(type);
    const float eps = static_cast<float>(number(a[3]));
    const OnDevice on(x);
    const Tensor y = x.out(a[4], type, "out");
    if (a[4] != Py_None) {
        check_apart(y, "out", x.t, x.rows, x.C, x.ld, "x");
        check_apart(y, "out", a[1], "gamma");
        check_apart(y, "out", a[2], "beta");
    }
    Tensor mean, rstd;
    const bool stats = a[6] == Py_True;
    if (stats) {
        mean = x.stat();
        rstd = x.stat();
    }
    check("dwc_layer_norm_fwd",
          dwc_layer_norm_fwd(x.t.data_ptr(), x.ld, w.p[0], w.p[1], w.type, eps, y.data_ptr(), fp(mean), fp(rstd), x.rows,
                             static_cast<int>(x.C), in, od, on.stream));
    return stats ? pack({&y, &mean, &rstd}) : wrap(y);
}

// (dy, x, mean, rstd, gamma, out, param_grads)
PyObject* layer_norm_bwd(PyObject* const* a) {
    const Rows x(tensor(a[1], "x"), "x");
    const Tensor& dy = tensor(a[0], "dy");
    const int64_t lddy = x.like(dy, "dy");
    const float *mean = x.given_stat(a[2], "mean"), *rstd = x.given_stat(a[3], "rstd");
    const Params w(x, a[4], Py_None);
    const dwc_dtype_t type = code_of(x.t.scalar_type()), dtype = code_of(dy.scalar_type());
    const OnDevice on(x);
    const Tensor dx = x.out(a[5], x.t.scalar_type(), "out");
    if (a[5] != Py_None) {
        check_apart(dx, "out", dy, x.rows, x.C, lddy, "dy");
        check_apart(dx, "out", x.t, x.rows, x.C, x.ld, "x");
        check_apart(dx, "out", a[2], "mean");
        check_apart(dx, "out", a[3], "rstd");
        check_apart(dx, "out", a[4], "gamma");
    }
    const ParamGrads g(x, a[6] == Py_True);
    check("dwc_layer_norm_bwd",
          dwc_layer_norm_bwd(dy.data_ptr(), lddy, x.t.data_ptr(), x.ld, mean, rstd, w.p[0], w.type, dx.data_ptr(), g.dg,
                             g.db, x.rows, static_cast<int>(x.C), type, dtype, g.w, g.bytes, on.stream));
    return pack({&dx, &g.dgamma, &g.dbeta});
}

// (x, p, seed, offset, out)
template <bool kBackward>
PyObject* dropout(PyObject* const* a) {
    const char* what = kBackward ? "dy" : "x";
    const Rows x(tensor(a[0], what), what);
    const Random rnd(x, a[1], a[2], a[3]);
    const dwc_dtype_t type = code_of(x.t.scalar_type());
    const OnDevice on(x);
    const Tensor y = x.out(a[4], x.t.scalar_type(), "out");
    if (a[4] != Py_None) {
        check_apart(y, "out", x.t, x.rows, x.C, x.ld, what);
        check_apart(y, "out", a[3], "offset");
    }
    const auto call = kBackward ? dwc_dropout_bwd : dwc_dropout_fwd;
    check(kBackward ? "dwc_dropout_bwd" : "dwc_dropout_fwd",
          call(x.t.data_ptr(), x.ld, y.data_ptr(), x.rows, static_cast<int>(x.C), rnd.p, rnd.seed, rnd.offset, rnd.step,
               type, on.stream));
    return wrap(y);
}

// (x, res, gamma, beta, eps, p, seed, offset, out, z, stats)
PyObject* add_layer_norm_fwd(PyObject* const* a) {
    const Rows x(tensor(a[0], "x"), "x");
    const Tensor& res = tensor(a[1], "res");
    const int64_t ldres = x.like(res, "res");
    const Params w(x, a[2], a[3]);
    const float eps = static_cast<float>(number(a[4]));
    const Random rnd(x, a[5], a[6], a[7]);
    const dwc_dtype_t type = code_of(x.t.scalar_type()), wide = code_of(res.scalar_type());
    const OnDevice on(x);
    const Tensor y = x.out(a[8], x.t.scalar_type(), "out"), z = x.out(a[9], res.scalar_type(), "z");
    for (int i = 8; i <= 9; ++i) {
        if (a[i] == Py_None) continue;
        const Tensor& o = i == 8 ? y : z;
        const char* what = i == 8 ? "out" : "z";
        check_apart(o, what, x.t, x.rows, x.C, x.ld, "x");
        check_apart(o, what, res, x.rows, x.C, ldres, "res");
        check_apart(o, what, a[2], "gamma");
        check_apart(o, what, a[3], "beta");
        check_apart(o, what, a[7], "offset");
    }
    if (a[8] != Py_None && a[9] != Py_None) check_apart(y, "out", z, x.rows, x.C, x.C, "z", false);
    Tensor mean, rstd;
    const bool stats = a[10] == Py_True;
    if (stats) {
        mean = x.stat();
        rstd = x.stat();
    }
    check("dwc_add_layer_norm_fwd",
          dwc_add_layer_norm_fwd(x.t.data_ptr(), x.ld, res.data_ptr(), ldres, rnd.p, rnd.seed, rnd.offset, rnd.step, w.p[0],
                                 w.p[1], w.type, eps, z.data_ptr(), y.data_ptr(), fp(mean), fp(rstd), x.rows,
                                 static_cast<int>(x.C), type, wide, on.stream));
    return stats ? pack({&y, &z, &mean, &rstd}) : pack({&y, &z});
}

// (dy, z, mean, rstd, gamma, dz, p, seed, offset, param_grads)
PyObject* add_layer_norm_bwd(PyObject* const* a) {
    const Rows z(tensor(a[1], "z"), "z");
    const Tensor& dy = tensor(a[0], "dy");
    const int64_t lddy = z.like(dy, "dy");
    int64_t lddz = z.C;
    const void* dz = nullptr;
    if (a[5] != Py_None) {
        const Tensor& t = tensor(a[5], "dz");
        TORCH_CHECK_VALUE(t.scalar_type() == z.t.scalar_type(), "dz must have z's dtype");
        lddz = z.like(t, "dz");
        dz = t.data_ptr();
    }
    const float *mean = z.given_stat(a[2], "mean"), *rstd = z.given_stat(a[3], "rstd");
    const Params w(z, a[4], Py_None);
    const Random rnd(z, a[6], a[7], a[8]);
    const dwc_dtype_t type = code_of(dy.scalar_type()), wide = code_of(z.t.scalar_type());
    const OnDevice on(z);
    const Tensor dres = z.out(Py_None, z.t.scalar_type(), "dres");
    // without dropout and conversion dx is dres
    const bool own = rnd.p != 0.0 || type != wide;
    const Tensor dx = own ? z.out(Py_None, dy.scalar_type(), "dx") : dres;
    const ParamGrads g(z, a[9] == Py_True);
    check("dwc_add_layer_norm_bwd",
          dwc_add_layer_norm_bwd(dy.data_ptr(), lddy, dz, lddz, z.t.data_ptr(), z.ld, mean, rstd, w.p[0], w.type, rnd.p,
                                 rnd.seed, rnd.offset, rnd.step, own ? dx.data_ptr() : nullptr, dres.data_ptr(), g.dg, g.db,
                                 z.rows, static_cast<int>(z.C), type, wide, g.w, g.bytes, on.stream));
    return pack({&dx, &dres, &g.dgamma, &g.dbeta});
}

// (tensor, name): the row stride a call would use
PyObject* stride_of(PyObject* const* a) {
    const char* what = PyUnicode_AsUTF8(a[1]);
    if (what == nullptr) return nullptr;
    const Tensor& t = tensor(a[0], what);
    TORCH_CHECK_VALUE(t.dim() >= 1, what, " must be [..., C]");
    return PyLong_FromLongLong(row_stride(t, what));
}

PyObject* set_error(PyObject* const* a) {
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

template <Fast f, int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<layer_norm_fwd, 7>("layer_norm_fwd"),
                           method<layer_norm_bwd, 7>("layer_norm_bwd"),
                           method<dropout<false>, 5>("dropout_fwd"),
                           method<dropout<true>, 5>("dropout_bwd"),
                           method<add_layer_norm_fwd, 11>("add_layer_norm_fwd"),
                           method<add_layer_norm_bwd, 10>("add_layer_norm_bwd"),
                           method<stride_of, 2>("row_stride"),
                           method<set_error, 1>("set_error"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_norm_host", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__norm_host() { return PyModule_Create(&g_module); }
