// dwc_norm_py.cpp -- host path of the norm, dropout and sequence operators for Python (CPython C API).
//
// Small calls are bound by the host: through ctypes and tensor attributes read one by one a
// backward pass cost 23 us of Python beside 13 us of GPU work.  Here the checks, the outputs'
// allocation (PyTorch's allocator, so memory belongs to the current stream or graph) and the
// call of the C ABI (include/dwc_norm.h) are one C++ function per operator.  Nothing is computed
// here and nothing is kept between calls.  norm.py documents the functions and handles `stream`.
#include "dwc_py.h"
#include "dwc_seq_py.h"

namespace {

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

// Vectors of C values of one type each, or None.
struct Vectors {
    const void* p[3] = {nullptr, nullptr, nullptr};
    dwc_dtype_t type = DWC_F32;
    Vectors(const Rows& x, std::initializer_list<std::pair<PyObject*, const char*>> list) {
        bool any = false;
        int i = -1;
        for (const auto& [o, what] : list) {
            ++i;
            if (o == Py_None) continue;
            const Tensor& t = tensor(o, what);
            TORCH_CHECK_VALUE(t.dim() == 1 && t.numel() == x.C && t.device() == x.t.device() && t.is_contiguous(), what,
                              " must hold ", x.C, " values on ", x.t.device(), " (got ", t.sizes(), " on ", t.device(), ")");
            const dwc_dtype_t c = code_of(t.scalar_type());
            TORCH_CHECK_VALUE(!any || c == type, "gamma_post, gamma_pre and scale must have one dtype");
            type = c;
            any = true;
            p[i] = t.data_ptr();
        }
    }
};

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
    const OnDevice on(x.t);
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
    const OnDevice on(x.t);
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
    const OnDevice on(x.t);
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
    const OnDevice on(x.t);
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
    const OnDevice on(z.t);
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

// A gate (rows x C of x's type) or None.
struct Gate {
    const void* p = nullptr;
    int64_t ld = 0;
    dwc_gate_t act;
    bool given;
    Gate(const Rows& x, PyObject* o, PyObject* kind) : act(gate_code(kind)), given(o != Py_None) {
        if (!given) return;
        const Tensor& t = tensor(o, "gate");
        TORCH_CHECK_VALUE(t.scalar_type() == x.t.scalar_type(), "gate must have x's dtype");
        ld = x.like(t, "gate");
        p = t.data_ptr();
    }
};

// (x, res, gamma_post, gamma_pre, gate, scale, alpha, act, eps, out, z, stats)
PyObject* block_norm_fwd(PyObject* const* a) {
    const Rows x(tensor(a[0], "x"), "x");
    const Tensor& res = tensor(a[1], "res");
    const int64_t ldres = x.like(res, "res");
    const Vectors w(x, {{a[2], "gamma_post"}, {a[3], "gamma_pre"}, {a[5], "scale"}});
    const Gate gate(x, a[4], a[7]);
    const float alpha = static_cast<float>(number(a[6])), eps = static_cast<float>(number(a[8]));
    const dwc_dtype_t type = code_of(x.t.scalar_type()), wide = code_of(res.scalar_type());
    const OnDevice on(x.t);
    const Tensor y = x.out(a[9], x.t.scalar_type(), "out"), z = x.out(a[10], res.scalar_type(), "z");
    for (int i = 9; i <= 10; ++i) {
        if (a[i] == Py_None) continue;
        const Tensor& o = i == 9 ? y : z;
        const char* what = i == 9 ? "out" : "z";
        check_apart(o, what, x.t, x.rows, x.C, x.ld, "x");
        check_apart(o, what, res, x.rows, x.C, ldres, "res");
        if (gate.given) check_apart(o, what, tensor(a[4], "gate"), x.rows, x.C, gate.ld, "gate");
        check_apart(o, what, a[2], "gamma_post");
        check_apart(o, what, a[3], "gamma_pre");
        check_apart(o, what, a[5], "scale");
    }
    if (a[9] != Py_None && a[10] != Py_None) check_apart(y, "out", z, x.rows, x.C, x.C, "z", false);
    Tensor post, pre;
    const bool stats = a[11] == Py_True;
    if (stats) {
        post = x.stat();
        pre = x.stat();
    }
    check("dwc_block_norm_fwd",
          dwc_block_norm_fwd(x.t.data_ptr(), x.ld, res.data_ptr(), ldres, gate.p, gate.ld, gate.act, w.p[0], w.p[1], w.p[2],
                             w.type, alpha, eps, z.data_ptr(), y.data_ptr(), fp(post), fp(pre), x.rows,
                             static_cast<int>(x.C), type, wide, on.stream));
    return stats ? pack({&y, &z, &post, &pre}) : pack({&y, &z});
}

// (dy, x, z, rstd_post, rstd_pre, gamma_post, gamma_pre, gate, scale, alpha, act, dz, param_grads)
PyObject* block_norm_bwd(PyObject* const* a) {
    const Rows x(tensor(a[1], "x"), "x");
    const Tensor &dy = tensor(a[0], "dy"), &z = tensor(a[2], "z");
    TORCH_CHECK_VALUE(dy.scalar_type() == x.t.scalar_type(), "dy must have x's dtype");
    const int64_t lddy = x.like(dy, "dy"), ldz = x.like(z, "z");
    int64_t lddz = x.C;
    const void* dz = nullptr;
    if (a[11] != Py_None) {
        const Tensor& t = tensor(a[11], "dz");
        TORCH_CHECK_VALUE(t.scalar_type() == z.scalar_type(), "dz must have z's dtype");
        lddz = x.like(t, "dz");
        dz = t.data_ptr();
    }
    const float *post = x.given_stat(a[3], "rstd_post"), *pre = x.given_stat(a[4], "rstd_pre");
    const Vectors w(x, {{a[5], "gamma_post"}, {a[6], "gamma_pre"}, {a[8], "scale"}});
    const Gate gate(x, a[7], a[10]);
    const float alpha = static_cast<float>(number(a[9]));
    const dwc_dtype_t type = code_of(x.t.scalar_type()), wide = code_of(z.scalar_type());
    const OnDevice on(x.t);
    const Tensor dx = x.out(Py_None, x.t.scalar_type(), "dx"), dres = x.out(Py_None, z.scalar_type(), "dres");
    Tensor dgate, ws, grads[3];
    if (gate.given) dgate = x.out(Py_None, x.t.scalar_type(), "dgate");
    size_t bytes = 0;
    if (a[12] == Py_True) {
        // (gradients of the parameters that the call has)
        const int at[3] = {5, 6, 8};
        bool any = false;
        for (int i = 0; i < 3; ++i) {
            if (a[at[i]] == Py_None) continue;
            grads[i] = new_tensor({x.C}, at::kFloat, x.t.device());
            any = true;
        }
        if (any) {
            bytes = dwc_block_norm_bwd_workspace_size(x.rows, static_cast<int>(x.C));
            ws = new_tensor({static_cast<int64_t>(bytes)}, at::kByte, x.t.device());
        }
    }
    check("dwc_block_norm_bwd",
          dwc_block_norm_bwd(dy.data_ptr(), lddy, dz, lddz, x.t.data_ptr(), x.ld, z.data_ptr(), ldz, gate.p, gate.ld,
                             gate.act, post, pre, w.p[0], w.p[1], w.p[2], w.type, alpha, dx.data_ptr(), dres.data_ptr(),
                             gate.p != nullptr ? dgate.data_ptr() : nullptr, fp(grads[0]), fp(grads[1]), fp(grads[2]),
                             x.rows, static_cast<int>(x.C), type, wide, ws.defined() ? ws.data_ptr() : nullptr, bytes,
                             on.stream));
    return pack({&dx, &dres, &dgate, &grads[0], &grads[1], &grads[2]});
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

PyMethodDef g_methods[] = {method<layer_norm_fwd, 7>("layer_norm_fwd"),
                           method<layer_norm_bwd, 7>("layer_norm_bwd"),
                           method<dropout<false>, 5>("dropout_fwd"),
                           method<dropout<true>, 5>("dropout_bwd"),
                           method<add_layer_norm_fwd, 11>("add_layer_norm_fwd"),
                           method<add_layer_norm_bwd, 10>("add_layer_norm_bwd"),
                           method<block_norm_fwd, 12>("block_norm_fwd"),
                           method<block_norm_bwd, 13>("block_norm_bwd"),
                           method<seq::causal_conv_fwd, 8>("causal_conv_fwd"),
                           method<seq::causal_conv_bwd, 9>("causal_conv_bwd"),
                           method<seq::causal_conv_step, 6>("causal_conv_step"),
                           method<seq::scan_fwd, 14>("selective_scan_fwd"),
                           method<seq::scan_bwd, 14>("selective_scan_bwd"),
                           method<seq::scan_step, 11>("selective_scan_step"),
                           method<stride_of, 2>("row_stride"),
                           method<set_error, 1>("set_error"),
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_norm_host", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__norm_host() { return PyModule_Create(&g_module); }
