// dwc_seq_api.cu -- the C ABI declared in include/dwc_seq.h: argument validation and launches.
#include <cstdint>
#include <initializer_list>

#include "../../include/dwc_seq.h"
#include "dwc_seq_host.h"

using namespace dwc;

namespace {

constexpr long long kMaxElems = 1LL << 40;
constexpr long long kMaxPositions = (1LL << 31) - 64;      // (kernels count to the end of a tile behind the last one)
constexpr int kMaxChannels = 1 << 20;
constexpr int kMaxTaps = 16;

bool known(dwc_dtype_t t) { return t == DWC_F32 || t == DWC_BF16 || t == DWC_F16; }
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

dwc_status_t first_error(std::initializer_list<dwc_status_t> list) {
    for (dwc_status_t s : list)
        if (s != DWC_OK) return s;
    return DWC_OK;
}

dwc_status_t map_cuda(cudaError_t err) {
    if (err == cudaSuccess) return DWC_OK;
    (void)cudaGetLastError();  // do not leave the failure to the next launch check
    return DWC_ERR_CUDA;
}

dwc_status_t check_seqs(const dwc_seqs_t& s, long long width) {
    if (s.count < 0 || s.length < 0) return DWC_ERR_INVALID_ARG;
    if (s.count == 0 && s.offsets != nullptr && s.length > 0) return DWC_ERR_INVALID_ARG;
    if (misaligned(s.offsets, 4)) return DWC_ERR_ALIGNMENT;
    const long long most = s.offsets != nullptr || s.count == 0 ? kMaxPositions : kMaxPositions / s.count;
    if (s.length > most) return DWC_ERR_UNSUPPORTED;
    const long long rows = s.offsets != nullptr ? s.length : s.count * s.length;
    // (the states and the parameter gradients' partial rows, one of each per sequence or piece, as well)
    if (rows > kMaxElems / width || s.count > kMaxElems / width) return DWC_ERR_UNSUPPORTED;
    return DWC_OK;
}
long long positions(const dwc_seqs_t& s) { return s.offsets != nullptr ? s.length : s.count * s.length; }

// A view of `width` values a position: null only where `optional` or there are no positions.
dwc_status_t check_view(const dwc_rows_t& v, const dwc_seqs_t& s, int bytes, bool optional) {
    if (v.data == nullptr) return optional || positions(s) == 0 ? DWC_OK : DWC_ERR_INVALID_ARG;
    if (v.row_stride < 0 || (s.offsets == nullptr && v.seq_stride < 0)) return DWC_ERR_INVALID_ARG;
    if (s.length > 0 && v.row_stride > kMaxElems / s.length) return DWC_ERR_UNSUPPORTED;
    if (s.offsets == nullptr && s.count > 0 && v.seq_stride > kMaxElems / s.count) return DWC_ERR_UNSUPPORTED;
    return misaligned(v.data, bytes) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

dwc_status_t check_out(const void* p, const dwc_seqs_t& s, int bytes, bool optional) {
    if (p == nullptr) return optional || positions(s) == 0 ? DWC_OK : DWC_ERR_INVALID_ARG;
    return misaligned(p, bytes) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

Seqs seqs_of(const dwc_seqs_t& s) { return Seqs{s.offsets, s.count, s.length}; }

RowsView view_of(const dwc_rows_t& v, const dwc_seqs_t& s, int bytes) {
    const bool one_row = positions(s) <= 1;
    const bool vec = v.data != nullptr && !misaligned(v.data, 8 * static_cast<size_t>(bytes)) &&
                     (one_row || ((s.length <= 1 || v.row_stride % 8 == 0) &&
                                  (s.offsets != nullptr || s.count <= 1 || v.seq_stride % 8 == 0)));
    return RowsView{v.data, s.offsets != nullptr ? 0 : v.seq_stride, v.row_stride, vec};
}

// ---- causal convolution

dwc_status_t check_conv(const dwc_causal_conv_t* c, bool step) {
    if (c == nullptr) return DWC_ERR_INVALID_ARG;
    if (c->C < 1 || c->K < 1 || !known(c->dtype) || !known(c->param_dtype)) return DWC_ERR_INVALID_ARG;
    if (c->act != DWC_GATE_NONE && c->act != DWC_GATE_SILU) return DWC_ERR_INVALID_ARG;
    if (c->K > kMaxTaps || c->C > kMaxChannels) return DWC_ERR_UNSUPPORTED;
    if (step && (c->seqs.length != 1 || c->seqs.offsets != nullptr)) return DWC_ERR_INVALID_ARG;
    const int bytes = elem_bytes(c->dtype), wide = elem_bytes(c->param_dtype);
    const dwc_status_t st = first_error({check_seqs(c->seqs, static_cast<long long>(c->C) * c->K),
                                         check_view(c->x, c->seqs, bytes, false)});
    if (st != DWC_OK) return st;
    if (c->w == nullptr && positions(c->seqs) > 0) return DWC_ERR_INVALID_ARG;
    return misaligned(c->w, wide) || misaligned(c->bias, wide) || misaligned(c->state, bytes) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

CausalConv conv_of(const dwc_causal_conv_t& c, dwc_stream_t stream) {
    CausalConv p{};
    p.seqs = seqs_of(c.seqs);
    p.C = c.C;
    p.K = c.K;
    p.silu = c.act == DWC_GATE_SILU;
    p.type = c.dtype;
    p.param_type = c.param_dtype;
    p.x = view_of(c.x, c.seqs, elem_bytes(c.dtype));
    p.w = c.w;
    p.bias = c.bias;
    p.state = c.state;
    p.stream = stream;
    return p;
}

size_t conv_workspace(const dwc_causal_conv_t& c) {
    const Seqs s = seqs_of(c.seqs);
    return static_cast<size_t>(causal_conv_bwd_slots(s, c.C)) * (c.K + 1) * c.C * sizeof(float);
}

// ---- scan

dwc_status_t check_scan(const dwc_scan_t* c, bool step) {
    if (c == nullptr) return DWC_ERR_INVALID_ARG;
    if (c->C < 1 || c->N < 1 || c->G < 1 || !known(c->dtype)) return DWC_ERR_INVALID_ARG;
    if (c->C % c->G != 0) return DWC_ERR_INVALID_ARG;
    if (c->N > kScanMaxStates || c->C > kMaxChannels) return DWC_ERR_UNSUPPORTED;
    if (step && (c->seqs.length != 1 || c->seqs.offsets != nullptr)) return DWC_ERR_INVALID_ARG;
    const int bytes = elem_bytes(c->dtype);
    const dwc_status_t st = first_error(
        {check_seqs(c->seqs, static_cast<long long>(c->C) * c->N), check_view(c->u, c->seqs, bytes, false),
         check_view(c->dt, c->seqs, bytes, false), check_view(c->z, c->seqs, bytes, true),
         check_view(c->b, c->seqs, bytes, false), check_view(c->c, c->seqs, bytes, false)});
    if (st != DWC_OK) return st;
    if (c->A == nullptr && positions(c->seqs) > 0) return DWC_ERR_INVALID_ARG;
    return misaligned(c->A, 4) || misaligned(c->D, 4) || misaligned(c->dt_bias, 4) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

Scan scan_of(const dwc_scan_t& c, dwc_stream_t stream) {
    const int bytes = elem_bytes(c.dtype);
    Scan p{};
    p.seqs = seqs_of(c.seqs);
    p.C = c.C;
    p.N = c.N;
    p.G = c.G;
    p.softplus = c.softplus != 0;
    p.type = c.dtype;
    p.u = view_of(c.u, c.seqs, bytes);
    p.dt = view_of(c.dt, c.seqs, bytes);
    p.z = view_of(c.z, c.seqs, bytes);
    p.b = view_of(c.b, c.seqs, bytes);
    p.c = view_of(c.c, c.seqs, bytes);
    p.A = c.A;
    p.D = c.D;
    p.dt_bias = c.dt_bias;
    p.stream = stream;
    return p;
}

#define DWC_BY_TYPE(fn, p)                              \
    switch ((p).type) {                                 \
        case kF32: return map_cuda(fn##_f32(p));        \
        case kBF16: return map_cuda(fn##_bf16(p));      \
        default: return map_cuda(fn##_f16(p));          \
    }

dwc_status_t scan_fwd(const Scan& p) { DWC_BY_TYPE(launch_scan_fwd, p) }
dwc_status_t scan_bwd(const Scan& p) { DWC_BY_TYPE(launch_scan_bwd, p) }

dwc_status_t check_workspace(const void* ws, size_t bytes, size_t need) {
    if (need == 0) return DWC_OK;
    if (ws == nullptr || bytes < need) return DWC_ERR_WORKSPACE;
    return misaligned(ws, 16) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

// Gradients of parameters where there is nothing to add up.
dwc_status_t zero(float* p, long long n, dwc_stream_t stream) {
    return p == nullptr ? DWC_OK : map_cuda(cudaMemsetAsync(p, 0, static_cast<size_t>(n) * sizeof(float), stream));
}

}  // namespace

extern "C" {

dwc_status_t dwc_zero_beside_sequences(const dwc_seqs_t* seqs, void* const* tensors, const long long* row_bytes,
                                       int count, dwc_stream_t stream) {
    if (seqs == nullptr || count < 0 || (count > 0 && (tensors == nullptr || row_bytes == nullptr))) return DWC_ERR_INVALID_ARG;
    if (count > 8) return DWC_ERR_UNSUPPORTED;
    ZeroBeside p{};
    p.seqs = seqs_of(*seqs);
    p.count = count;
    p.stream = stream;
    for (int i = 0; i < count; ++i) {
        if (tensors[i] == nullptr || row_bytes[i] < 0) return DWC_ERR_INVALID_ARG;
        if (misaligned(tensors[i], 2) || row_bytes[i] % 2 != 0) return DWC_ERR_ALIGNMENT;
        const dwc_status_t st = check_seqs(*seqs, row_bytes[i] < 1 ? 1 : row_bytes[i]);
        if (st != DWC_OK) return st;
        p.p[i] = tensors[i];
        p.halves[i] = row_bytes[i] / 2;
    }
    if (seqs->offsets == nullptr || seqs->length == 0 || count == 0) return DWC_OK;
    return map_cuda(launch_zero_beside(p));
}

dwc_status_t dwc_causal_conv_fwd(const dwc_causal_conv_t* conv, void* y, void* final_state, dwc_stream_t stream) {
    dwc_status_t st = check_conv(conv, false);
    if (st != DWC_OK) return st;
    const int bytes = elem_bytes(conv->dtype);
    st = first_error({check_out(y, conv->seqs, bytes, false), check_out(final_state, conv->seqs, bytes, true)});
    if (st != DWC_OK) return st;
    if (conv->K == 1) final_state = nullptr;
    if (conv->seqs.count == 0 || (positions(conv->seqs) == 0 && final_state == nullptr)) return DWC_OK;
    if (conv->w == nullptr) return DWC_ERR_INVALID_ARG;
    CausalConv p = conv_of(*conv, stream);
    p.y = y;
    p.final_state = final_state;
    return map_cuda(launch_causal_conv_fwd(p));
}

size_t dwc_causal_conv_bwd_workspace_size(const dwc_causal_conv_t* conv) {
    return check_conv(conv, false) == DWC_OK ? conv_workspace(*conv) : 0;
}

dwc_status_t dwc_causal_conv_bwd(const dwc_causal_conv_t* conv, const dwc_rows_t* dy, const void* dfinal, void* dx,
                                 void* dstate, float* dw, float* dbias, void* workspace, size_t workspace_bytes,
                                 dwc_stream_t stream) {
    dwc_status_t st = check_conv(conv, false);
    if (st != DWC_OK) return st;
    if (dy == nullptr) return DWC_ERR_INVALID_ARG;
    const int bytes = elem_bytes(conv->dtype);
    st = first_error({check_view(*dy, conv->seqs, bytes, false), check_out(dx, conv->seqs, bytes, false),
                      check_out(dstate, conv->seqs, bytes, true), check_out(dfinal, conv->seqs, bytes, true)});
    if (st != DWC_OK) return st;
    if (misaligned(dw, 4) || misaligned(dbias, 4)) return DWC_ERR_ALIGNMENT;
    if (conv->K == 1) dstate = nullptr, dfinal = nullptr;
    if (conv->seqs.count == 0 || (positions(conv->seqs) == 0 && dstate == nullptr))
        return first_error({zero(dw, static_cast<long long>(conv->K) * conv->C, stream), zero(dbias, conv->C, stream)});
    if (conv->w == nullptr) return DWC_ERR_INVALID_ARG;
    CausalConv p = conv_of(*conv, stream);
    if (dw != nullptr || dbias != nullptr) {
        st = check_workspace(workspace, workspace_bytes, conv_workspace(*conv));
        if (st != DWC_OK) return st;
        p.partial = static_cast<float*>(workspace);
    }
    p.dy = view_of(*dy, conv->seqs, bytes);
    p.dfinal = dfinal;
    p.dx = dx;
    p.dstate = dstate;
    p.dw = dw;
    p.dbias = dbias;
    return map_cuda(launch_causal_conv_bwd(p));
}

dwc_status_t dwc_causal_conv_step(const dwc_causal_conv_t* conv, void* state, long long state_stride, void* y,
                                  dwc_stream_t stream) {
    dwc_status_t st = check_conv(conv, true);
    if (st != DWC_OK) return st;
    const int bytes = elem_bytes(conv->dtype);
    st = first_error({check_out(y, conv->seqs, bytes, false), check_out(state, conv->seqs, bytes, conv->K == 1)});
    if (st != DWC_OK) return st;
    const long long held = static_cast<long long>(conv->K - 1) * conv->C;
    if (conv->seqs.count > 1 && state_stride < held) return DWC_ERR_INVALID_ARG;
    if (conv->seqs.count > 0 && state_stride > kMaxElems / conv->seqs.count) return DWC_ERR_UNSUPPORTED;
    if (conv->seqs.count == 0) return DWC_OK;
    CausalConv p = conv_of(*conv, stream);
    p.y = y;
    return map_cuda(launch_causal_conv_step(p, state, state_stride));
}

size_t dwc_selective_scan_saved_floats(const dwc_scan_t* scan) {
    if (check_scan(scan, false) != DWC_OK) return 0;
    return static_cast<size_t>(seq_slots(seqs_of(scan->seqs), kScanTile)) * scan->C * scan->N;
}

size_t dwc_selective_scan_fwd_workspace_size(const dwc_scan_t* scan) {
    if (check_scan(scan, false) != DWC_OK || scan->seqs.count == 0) return 0;
    Scan p = scan_of(*scan, nullptr);
    p.span = scan_fwd_span(p);
    return scan_fwd_workspace_floats(p) * sizeof(float);
}

size_t dwc_selective_scan_bwd_workspace_size(const dwc_scan_t* scan) {
    if (check_scan(scan, false) != DWC_OK || scan->seqs.count == 0) return 0;
    Scan p = scan_of(*scan, nullptr);
    p.span = scan_bwd_span(p);
    return scan_bwd_workspace_floats(p) * sizeof(float);
}

dwc_status_t dwc_selective_scan_fwd(const dwc_scan_t* scan, const float* state, void* y, float* final_state,
                                    float* saved, void* workspace, size_t workspace_bytes, dwc_stream_t stream) {
    dwc_status_t st = check_scan(scan, false);
    if (st != DWC_OK) return st;
    st = check_out(y, scan->seqs, elem_bytes(scan->dtype), false);
    if (st != DWC_OK) return st;
    if (misaligned(state, 4) || misaligned(final_state, 4) || misaligned(saved, 4)) return DWC_ERR_ALIGNMENT;
    if (scan->seqs.count == 0 || (positions(scan->seqs) == 0 && final_state == nullptr)) return DWC_OK;
    if (scan->A == nullptr) return DWC_ERR_INVALID_ARG;
    Scan p = scan_of(*scan, stream);
    p.span = scan_fwd_span(p);
    st = check_workspace(workspace, workspace_bytes, scan_fwd_workspace_floats(p) * sizeof(float));
    if (st != DWC_OK) return st;
    p.state = state;
    p.y = y;
    p.final_state = final_state;
    p.saved = saved;
    p.workspace = static_cast<float*>(workspace);
    return scan_fwd(p);
}

dwc_status_t dwc_selective_scan_bwd(const dwc_scan_t* scan, const dwc_rows_t* dy, const float* saved,
                                    const float* dfinal, void* du, void* ddt, void* dz, void* db, void* dc, float* dA,
                                    float* dD, float* ddt_bias, float* dstate, void* workspace,
                                    size_t workspace_bytes, dwc_stream_t stream) {
    dwc_status_t st = check_scan(scan, false);
    if (st != DWC_OK) return st;
    if (dy == nullptr || dA == nullptr || dD == nullptr || ddt_bias == nullptr) return DWC_ERR_INVALID_ARG;
    const int bytes = elem_bytes(scan->dtype);
    st = first_error({check_view(*dy, scan->seqs, bytes, false), check_out(saved, scan->seqs, 4, false),
                      check_out(du, scan->seqs, bytes, false), check_out(ddt, scan->seqs, bytes, false),
                      check_out(dz, scan->seqs, bytes, scan->z.data == nullptr), check_out(db, scan->seqs, bytes, false),
                      check_out(dc, scan->seqs, bytes, false)});
    if (st != DWC_OK) return st;
    if (misaligned(dfinal, 4) || misaligned(dA, 4) || misaligned(dD, 4) || misaligned(ddt_bias, 4) || misaligned(dstate, 4))
        return DWC_ERR_ALIGNMENT;
    if (scan->seqs.count == 0 || (positions(scan->seqs) == 0 && dstate == nullptr))
        return first_error({zero(dA, static_cast<long long>(scan->C) * scan->N, stream), zero(dD, scan->C, stream),
                            zero(ddt_bias, scan->C, stream)});
    if (scan->A == nullptr) return DWC_ERR_INVALID_ARG;
    Scan p = scan_of(*scan, stream);
    p.span = scan_bwd_span(p);
    st = check_workspace(workspace, workspace_bytes, scan_bwd_workspace_floats(p) * sizeof(float));
    if (st != DWC_OK) return st;
    p.dy = view_of(*dy, scan->seqs, bytes);
    p.saved = const_cast<float*>(saved);
    p.dfinal = dfinal;
    p.du = du;
    p.ddt = ddt;
    p.dz = dz;
    p.db = db;
    p.dc = dc;
    p.dA = dA;
    p.dD = dD;
    p.ddt_bias = ddt_bias;
    p.dstate = dstate;
    p.workspace = static_cast<float*>(workspace);
    return scan_bwd(p);
}

dwc_status_t dwc_selective_scan_step(const dwc_scan_t* scan, float* state, long long state_stride, void* y,
                                     dwc_stream_t stream) {
    dwc_status_t st = check_scan(scan, true);
    if (st != DWC_OK) return st;
    st = first_error({check_out(y, scan->seqs, elem_bytes(scan->dtype), false), check_out(state, scan->seqs, 4, false)});
    if (st != DWC_OK) return st;
    const long long held = static_cast<long long>(scan->C) * scan->N;
    if (scan->seqs.count > 1 && state_stride < held) return DWC_ERR_INVALID_ARG;
    if (scan->seqs.count > 0 && state_stride > kMaxElems / scan->seqs.count) return DWC_ERR_UNSUPPORTED;
    if (scan->seqs.count == 0) return DWC_OK;
    Scan p = scan_of(*scan, stream);
    p.y = y;
    return map_cuda(launch_scan_step(p, state, state_stride));
}

}  // extern "C"
