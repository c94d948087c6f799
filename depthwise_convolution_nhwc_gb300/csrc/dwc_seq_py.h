// dwc_seq_py.h -- host path of the sequence operators for Python: checks, output allocation and the
// library call (include/dwc_seq.h) as one function each.  seq.py documents them.
#pragma once

#include "dwc_py.h"

namespace {
namespace seq {

// The tensor whose shape, sequences and device a call goes by: [B, T, C], with `offsets` [L, C], and
// for one position of each sequence [B, C].
struct Input {
    const Tensor& t;
    int lead;                  // leading axes
    int64_t C;
    dwc_seqs_t seqs{};
    Input(PyObject* o, const char* what, PyObject* offsets, bool step = false) : t(tensor(o, what)) {
        TORCH_CHECK_VALUE(t.is_cuda(), "tensors must be on a CUDA device (no CPU fallback)");
        const bool packed = !step && offsets != Py_None;
        lead = step || packed ? 1 : 2;
        TORCH_CHECK_VALUE(t.dim() == lead + 1 && t.size(-1) >= 1, what, " must be ",
                          step ? "[B, C]" : packed ? "[rows, C] with offsets" : "[B, T, C]", " (got ", t.sizes(), ")");
        C = t.size(-1);
        TORCH_CHECK_VALUE(C <= INT32_MAX && t.size(0) <= INT32_MAX, what, " is larger than the library takes");
        if (packed) {
            const Tensor& f = tensor(offsets, "offsets");
            TORCH_CHECK_VALUE(f.dim() == 1 && f.numel() >= 1 && f.scalar_type() == at::kInt && f.device() == t.device() &&
                                  f.is_contiguous(),
                              "offsets must be a contiguous int32 vector on ", t.device(), " (got ", f.sizes(), " ",
                              f.scalar_type(), " on ", f.device(), ")");
            TORCH_CHECK_VALUE(f.numel() - 1 <= INT32_MAX, "offsets has more entries than the library takes");
            seqs = {static_cast<int>(f.numel() - 1), t.size(0), static_cast<const int*>(f.data_ptr())};
        } else {
            seqs = {static_cast<int>(t.size(0)), step ? 1 : t.size(1), nullptr};
        }
    }
    at::IntArrayRef leading() const { return t.sizes().slice(0, lead); }
    // a view of this tensor's positions whose last axes are `width` adjacent values
    dwc_rows_t rows(const Tensor& v) const {
        const auto stride = [&](int i) { return v.size(i) == 1 ? int64_t{0} : v.stride(i); };
        if (lead == 1) return seqs.offsets != nullptr ? dwc_rows_t{v.data_ptr(), 0, stride(0)} : dwc_rows_t{v.data_ptr(), stride(0), 0};
        return {v.data_ptr(), stride(0), stride(1)};
    }
    dwc_rows_t own(const char* what) const {
        TORCH_CHECK_VALUE(C == 1 || t.stride(-1) == 1 || t.numel() == 0, what, ": channels must be adjacent (stride ", t.stride(-1), ")");
        return rows(t);
    }
    // an input of this tensor's shape and type
    dwc_rows_t like(PyObject* o, const char* what, bool optional = false) const {
        if (optional && o == Py_None) return {nullptr, 0, 0};
        const Tensor& v = tensor(o, what);
        TORCH_CHECK_VALUE(v.sizes() == t.sizes() && v.device() == t.device(), what, " must be a ", t.sizes(), " tensor on ",
                          t.device(), " (got ", v.sizes(), " on ", v.device(), ")");
        TORCH_CHECK_VALUE(v.scalar_type() == t.scalar_type(), what, " must be ", t.scalar_type(), " (got ", v.scalar_type(), ")");
        TORCH_CHECK_VALUE(C == 1 || v.stride(-1) == 1 || v.numel() == 0, what, ": channels must be adjacent (stride ", v.stride(-1), ")");
        return rows(v);
    }
    // B or C of a scan: the leading axes, then [G, N] or [N]
    dwc_rows_t states(PyObject* o, const char* what, int64_t N, int64_t& G) const {
        const Tensor& v = tensor(o, what);
        const bool grouped = v.dim() == lead + 2;
        TORCH_CHECK_VALUE((grouped || v.dim() == lead + 1) && v.sizes().slice(0, lead) == leading() && v.size(-1) == N &&
                              v.device() == t.device() && v.scalar_type() == t.scalar_type(),
                          what, " must be ", leading(), " x groups x ", N, " of ", t.scalar_type(), " on ", t.device(), " (got ",
                          v.sizes(), " ", v.scalar_type(), " on ", v.device(), ")");
        G = grouped ? v.size(-2) : 1;
        TORCH_CHECK_VALUE(v.numel() == 0 || ((N == 1 || v.stride(-1) == 1) && (G <= 1 || v.stride(-2) == N)), what,
                          ": the groups' states must be adjacent (strides ", v.strides(), ")");
        return rows(v);
    }
    Tensor make(at::IntArrayRef shape, ScalarType type) const { return new_tensor(shape, type, t.device()); }
    Tensor make() const { return make(t.sizes(), t.scalar_type()); }
    // a dense output of this tensor's shape: the caller's, apart from the call's inputs, or a new one
    Tensor out(PyObject* o, const char* what, std::initializer_list<PyObject*> inputs) const {
        if (o == Py_None) return make();
        const Tensor& v = tensor(o, what);
        TORCH_CHECK_VALUE(v.sizes() == t.sizes() && v.scalar_type() == t.scalar_type() && v.device() == t.device() &&
                              v.is_contiguous(),
                          what, " must be a contiguous ", t.sizes(), " ", t.scalar_type(), " tensor on ", t.device(), " (got ",
                          v.sizes(), " ", v.scalar_type(), " on ", v.device(), ")");
        apart(v, what, inputs);
        return v;
    }
    // an fp32 tensor of a given shape, dense
    const float* floats(PyObject* o, const char* what, at::IntArrayRef shape, bool optional = true) const {
        return static_cast<const float*>(dense(o, what, shape, at::kFloat, optional));
    }
    const void* dense(PyObject* o, const char* what, at::IntArrayRef shape, ScalarType type, bool optional) const {
        if (optional && o == Py_None) return nullptr;
        const Tensor& v = tensor(o, what);
        TORCH_CHECK_VALUE(v.sizes() == shape && v.scalar_type() == type && v.device() == t.device() && v.is_contiguous(), what,
                          " must be a contiguous ", shape, " ", type, " tensor on ", t.device(), " (got ", v.sizes(), " ",
                          v.scalar_type(), " on ", v.device(), ")");
        return v.data_ptr();
    }
    // a state updated in place: [B, ...] whose entries are dense, one stride between them
    void* state(PyObject* o, const char* what, at::IntArrayRef shape, ScalarType type, int64_t& stride,
                std::initializer_list<PyObject*> others) const {
        const Tensor& v = tensor(o, what);
        TORCH_CHECK_VALUE(v.sizes() == shape && v.scalar_type() == type && v.device() == t.device(), what, " must be a ", shape,
                          " ", type, " tensor on ", t.device(), " (got ", v.sizes(), " ", v.scalar_type(), " on ", v.device(), ")");
        const int64_t held = shape[1] * shape[2];
        stride = shape[0] > 1 ? v.stride(0) : held;
        TORCH_CHECK_VALUE(v.numel() == 0 || ((shape[2] == 1 || v.stride(2) == 1) && (shape[1] == 1 || v.stride(1) == shape[2]) &&
                                             stride >= held),
                          what, ": each sequence's state must be dense and apart from the others (strides ", v.strides(), ")");
        apart(v, what, others);
        return v.data_ptr();
    }

    // `out` must not share memory with a call's other tensors.  Of the ranges of addresses that meet, those are apart whose
    // entries along the first axis interleave: a sequence's state and its next input side by side in a row of one cache.
    struct Reach {
        int64_t entries, stride, bytes;        // of an entry: from its first element to its last
        uintptr_t lo;
        explicit Reach(const Tensor& v) : entries(1), stride(0), bytes(1), lo(reinterpret_cast<uintptr_t>(v.data_ptr())) {
            const bool several = v.dim() > 0 && v.size(0) > 1 && v.stride(0) > 0;
            for (int64_t i = several ? 1 : 0; i < v.dim(); ++i) bytes += (v.size(i) - 1) * v.stride(i);
            bytes *= v.element_size();
            if (several) entries = v.size(0), stride = v.stride(0) * v.element_size();
        }
        uintptr_t end() const { return lo + (entries - 1) * stride + bytes; }
    };
    static bool interleave(const Reach& a, const Reach& b) {
        const int64_t stride = a.entries > 1 ? a.stride : b.stride;
        if (stride <= 0 || (a.entries > 1 && b.entries > 1 && a.stride != b.stride)) return false;
        // from the start of an entry of `a` to the next start of one of `b`, and the room behind that
        const int64_t off = static_cast<int64_t>(b.lo - a.lo) % stride, ahead = off < 0 ? off + stride : off;
        return ahead >= a.bytes && ahead + b.bytes <= stride;
    }
    static void apart(const Tensor& out, const char* what, std::initializer_list<PyObject*> others) {
        if (out.numel() == 0) return;
        const Reach mine(out);
        for (PyObject* o : others) {
            if (o == nullptr || !THPVariable_Check(o)) continue;
            const Tensor& v = THPVariable_Unpack(o);
            if (v.numel() == 0) continue;
            const Reach theirs(v);
            TORCH_CHECK_VALUE(theirs.end() <= mine.lo || theirs.lo >= mine.end() || interleave(mine, theirs), what,
                              " overlaps another tensor of the call");
        }
    }
};

// Packed rows in front of the first and behind the last sequence of new outputs.
void zero_beside(const Input& x, dwc_stream_t stream, std::initializer_list<const Tensor*> list) {
    if (x.seqs.offsets == nullptr) return;
    void* data[8];
    long long bytes[8];
    int n = 0;
    for (const Tensor* t : list) {
        if (!t->defined() || t->numel() == 0) continue;
        data[n] = t->data_ptr();
        bytes[n++] = t->numel() / t->size(0) * t->element_size();
    }
    check("dwc_zero_beside_sequences", dwc_zero_beside_sequences(&x.seqs, data, bytes, n, stream));
}

// ---- causal convolution

struct Conv {
    dwc_causal_conv_t c{};
    int64_t held[3];           // shape of the states
    Conv(const Input& x, PyObject* w_, PyObject* bias_, PyObject* act, PyObject* state) {
        const Tensor& w = tensor(w_, "w");
        TORCH_CHECK_VALUE(w.dim() == 2 && w.size(0) >= 1 && w.size(1) == x.C && w.device() == x.t.device() && w.is_contiguous(),
                          "w must be a contiguous [taps, ", x.C, "] tensor on ", x.t.device(), " (got ", w.sizes(), " on ",
                          w.device(), ")");
        TORCH_CHECK_VALUE(w.size(0) <= INT32_MAX, "w has more taps than the library takes");
        c.seqs = x.seqs;
        c.C = static_cast<int>(x.C);
        c.K = static_cast<int>(w.size(0));
        c.act = gate_code(act);
        TORCH_CHECK_VALUE(c.act != DWC_GATE_SIGMOID, "act must be \"none\" or \"silu\"");
        c.dtype = code_of(x.t.scalar_type());
        c.param_dtype = code_of(w.scalar_type());
        c.w = w.data_ptr();
        const int64_t channels[1] = {x.C};
        c.bias = x.dense(bias_, "bias", channels, w.scalar_type(), true);
        held[0] = x.seqs.count, held[1] = c.K - 1, held[2] = x.C;
        c.state = x.dense(state, "state", held, x.t.scalar_type(), true);
        c.x = x.own("x");
    }
};

// (x, w, bias, act, state, offsets, out, final)
PyObject* causal_conv_fwd(PyObject* const* a) {
    const Input x(a[0], "x", a[5]);
    const Conv conv(x, a[1], a[2], a[3], a[4]);
    const OnDevice on(x.t);
    const Tensor y = x.out(a[6], "out", {a[0], a[1], a[2], a[4], a[5]});
    Tensor last;
    if (a[7] == Py_True) last = x.make(conv.held, x.t.scalar_type());
    check("dwc_causal_conv_fwd",
          dwc_causal_conv_fwd(&conv.c, y.data_ptr(), last.defined() ? last.data_ptr() : nullptr, on.stream));
    if (a[6] == Py_None) zero_beside(x, on.stream, {&y});
    return last.defined() ? pack({&y, &last}) : wrap(y);
}

// (dy, x, w, bias, act, state, offsets, dfinal, param_grads)
PyObject* causal_conv_bwd(PyObject* const* a) {
    const Input x(a[1], "x", a[6]);
    const Conv conv(x, a[2], a[3], a[4], a[5]);
    const dwc_rows_t dy = x.like(a[0], "dy");
    const void* dfinal = x.dense(a[7], "dfinal", conv.held, x.t.scalar_type(), true);
    const OnDevice on(x.t);
    const Tensor dx = x.make();
    Tensor dstate, dw, dbias, ws;
    if (a[5] != Py_None) dstate = x.make(conv.held, x.t.scalar_type());
    size_t bytes = 0;
    if (a[8] == Py_True) {
        dw = x.make({conv.c.K, x.C}, at::kFloat);
        if (a[3] != Py_None) dbias = x.make({x.C}, at::kFloat);
        bytes = dwc_causal_conv_bwd_workspace_size(&conv.c);
        ws = x.make({static_cast<int64_t>(bytes)}, at::kByte);
    }
    check("dwc_causal_conv_bwd",
          dwc_causal_conv_bwd(&conv.c, &dy, dfinal, dx.data_ptr(), dstate.defined() ? dstate.data_ptr() : nullptr, fp(dw),
                              fp(dbias), ws.defined() ? ws.data_ptr() : nullptr, bytes, on.stream));
    zero_beside(x, on.stream, {&dx});
    return pack({&dx, &dw, &dbias, &dstate});
}

// (x, state, w, bias, act, out)
PyObject* causal_conv_step(PyObject* const* a) {
    const Input x(a[0], "x", Py_None, true);
    const Conv conv(x, a[2], a[3], a[4], Py_None);
    int64_t stride;
    void* state = x.state(a[1], "state", conv.held, x.t.scalar_type(), stride, {a[0], a[2], a[3], a[5]});
    const OnDevice on(x.t);
    const Tensor y = x.out(a[5], "out", {a[0], a[2], a[3]});
    check("dwc_causal_conv_step", dwc_causal_conv_step(&conv.c, state, stride, y.data_ptr(), on.stream));
    return wrap(y);
}

// ---- selective scan

struct ScanArgs {
    dwc_scan_t s{};
    int64_t held[3];           // shape of the states
    bool grouped;              // B and C have an axis of groups
    // u, dt, A, B, C, D, z, dt_bias, softplus
    ScanArgs(const Input& u, PyObject* dt, PyObject* A_, PyObject* B, PyObject* C, PyObject* D, PyObject* z, PyObject* bias,
             PyObject* softplus) {
        const Tensor& A = tensor(A_, "A");
        TORCH_CHECK_VALUE(A.dim() == 2 && A.size(0) == u.C && A.size(1) >= 1 && A.size(1) <= INT32_MAX &&
                              A.scalar_type() == at::kFloat && A.device() == u.t.device() && A.is_contiguous(),
                          "A must be a contiguous fp32 [", u.C, ", states] tensor on ", u.t.device(), " (got ", A.sizes(), " ",
                          A.scalar_type(), " on ", A.device(), ")");
        const int64_t N = A.size(1);
        int64_t G = 1, G2 = 1;
        s.seqs = u.seqs;
        s.C = static_cast<int>(u.C);
        s.N = static_cast<int>(N);
        s.softplus = softplus == Py_True;
        s.dtype = code_of(u.t.scalar_type());
        s.u = u.own("u");
        s.dt = u.like(dt, "dt");
        s.z = u.like(z, "z", true);
        s.b = u.states(B, "B", N, G);
        s.c = u.states(C, "C", N, G2);
        TORCH_CHECK_VALUE(G == G2 && tensor(B, "B").dim() == tensor(C, "C").dim(), "B and C must have one shape");
        TORCH_CHECK_VALUE(G >= 1 && u.C % G == 0, "the groups of B and C must divide the ", u.C, " channels (got ", G, ")");
        grouped = tensor(B, "B").dim() == u.lead + 2;
        s.G = static_cast<int>(G);
        const int64_t channels[1] = {u.C};
        s.A = static_cast<const float*>(A.data_ptr());
        s.D = u.floats(D, "D", channels);
        s.dt_bias = u.floats(bias, "dt_bias", channels);
        held[0] = u.seqs.count, held[1] = u.C, held[2] = N;
    }
};

// (u, dt, A, B, C, D, z, dt_bias, softplus, state, offsets, out, final, save)
PyObject* scan_fwd(PyObject* const* a) {
    const Input u(a[0], "u", a[10]);
    const ScanArgs scan(u, a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
    const float* state = u.floats(a[9], "state", scan.held);
    const OnDevice on(u.t);
    const Tensor y = u.out(a[11], "out", {a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[9], a[10]});
    Tensor last, saved, ws;
    if (a[12] == Py_True) last = u.make(scan.held, at::kFloat);
    if (a[13] == Py_True)
        saved = u.make({static_cast<int64_t>(dwc_selective_scan_saved_floats(&scan.s)) / (u.C * scan.s.N), u.C, scan.s.N}, at::kFloat);
    const size_t bytes = dwc_selective_scan_fwd_workspace_size(&scan.s);
    if (bytes > 0) ws = u.make({static_cast<int64_t>(bytes)}, at::kByte);
    check("dwc_selective_scan_fwd",
          dwc_selective_scan_fwd(&scan.s, state, y.data_ptr(), fp(last), fp(saved), ws.defined() ? ws.data_ptr() : nullptr,
                                 bytes, on.stream));
    if (a[11] == Py_None) zero_beside(u, on.stream, {&y});
    if (last.defined() && saved.defined()) return pack({&y, &last, &saved});
    return last.defined() ? pack({&y, &last}) : saved.defined() ? pack({&y, &saved}) : wrap(y);
}

// (dy, u, dt, A, B, C, saved, D, z, dt_bias, softplus, offsets, dfinal, state_grad)
PyObject* scan_bwd(PyObject* const* a) {
    const Input u(a[1], "u", a[11]);
    const ScanArgs scan(u, a[2], a[3], a[4], a[5], a[7], a[8], a[9], a[10]);
    const dwc_rows_t dy = u.like(a[0], "dy");
    const int64_t slots = static_cast<int64_t>(dwc_selective_scan_saved_floats(&scan.s)) / (u.C * scan.s.N);
    const int64_t kept[3] = {slots, u.C, scan.s.N};
    const float* saved = u.floats(a[6], "saved", kept, false);
    const float* dfinal = u.floats(a[12], "dfinal", scan.held);
    const OnDevice on(u.t);
    const Tensor du = u.make(), ddt = u.make();
    const Tensor db = u.make(tensor(a[4], "B").sizes(), u.t.scalar_type()), dc = u.make(db.sizes(), u.t.scalar_type());
    const Tensor dA = u.make({u.C, scan.s.N}, at::kFloat), dD = u.make({u.C}, at::kFloat), dbias = u.make({u.C}, at::kFloat);
    Tensor dz, dstate;
    if (a[8] != Py_None) dz = u.make();
    if (a[13] == Py_True) dstate = u.make(scan.held, at::kFloat);
    const size_t bytes = dwc_selective_scan_bwd_workspace_size(&scan.s);
    const Tensor ws = u.make({static_cast<int64_t>(bytes)}, at::kByte);
    check("dwc_selective_scan_bwd",
          dwc_selective_scan_bwd(&scan.s, &dy, saved, dfinal, du.data_ptr(), ddt.data_ptr(),
                                 dz.defined() ? dz.data_ptr() : nullptr, db.data_ptr(), dc.data_ptr(), fp(dA), fp(dD),
                                 fp(dbias), fp(dstate), ws.data_ptr(), bytes, on.stream));
    zero_beside(u, on.stream, {&du, &ddt, &dz, &db, &dc});
    const Tensor none;
    return pack({&du, &ddt, &dA, &db, &dc, a[7] != Py_None ? &dD : &none, &dz, a[9] != Py_None ? &dbias : &none, &dstate});
}

// (u, dt, A, B, C, state, D, z, dt_bias, softplus, out)
PyObject* scan_step(PyObject* const* a) {
    const Input u(a[0], "u", Py_None, true);
    const ScanArgs scan(u, a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[9]);
    int64_t stride;
    auto* state = static_cast<float*>(u.state(a[5], "state", scan.held, at::kFloat, stride,
                                              {a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[10]}));
    const OnDevice on(u.t);
    const Tensor y = u.out(a[10], "out", {a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8]});
    check("dwc_selective_scan_step", dwc_selective_scan_step(&scan.s, state, stride, y.data_ptr(), on.stream));
    return wrap(y);
}

}  // namespace seq
}  // namespace
