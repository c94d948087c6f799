// dwc_norm_api.cu -- the C ABI declared in include/dwc_norm.h: argument validation and the choice
// between the kernels.
#include <cmath>
#include <cstdint>

#include "../../include/dwc_norm.h"
#include "dwc_norm_host.h"

using namespace dwc;

namespace {

constexpr long long kMaxElems = 1LL << 40;
constexpr int kMaxChannels = 1 << 24;

bool known(dwc_dtype_t t) { return t == DWC_F32 || t == DWC_BF16 || t == DWC_F16; }

// A stream of `wide` with branches of `narrow`: the same type, or an fp32 stream.
bool valid_pair(dwc_dtype_t wide, dwc_dtype_t narrow) {
    return known(wide) && known(narrow) && (wide == narrow || wide == DWC_F32);
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

dwc_status_t check_rows(long long rows, int C) {
    if (rows < 0 || C < 1) return DWC_ERR_INVALID_ARG;
    if (C > kMaxChannels || rows > kMaxElems / C) return DWC_ERR_UNSUPPORTED;
    return DWC_OK;
}

// A tensor argument of `rows` rows: null only where `optional` or there are no rows.
dwc_status_t check_tensor(const void* p, long long ld, long long rows, int C, int bytes, bool optional) {
    if (p == nullptr) return optional || rows == 0 ? DWC_OK : DWC_ERR_INVALID_ARG;
    if (ld < C) return DWC_ERR_INVALID_ARG;
    if (rows > 0 && ld > kMaxElems / rows) return DWC_ERR_UNSUPPORTED;
    return misaligned(p, bytes) ? DWC_ERR_ALIGNMENT : DWC_OK;
}

// Whether `out` (dense, `out_type`) is the input `in`.  An update in place reads each element before it is
// overwritten; another type or row stride would overwrite elements that are still to be read.
dwc_status_t check_in_place(const void* out, int out_type, const void* in, long long ld, int type, long long rows,
                            int C, bool& in_place) {
    if (out == nullptr || out != in || rows == 0) return DWC_OK;
    in_place = true;
    return out_type == type && (ld == C || rows == 1) ? DWC_OK : DWC_ERR_INVALID_ARG;
}

// The first error of a list of checks.
dwc_status_t first_error(std::initializer_list<dwc_status_t> list) {
    for (dwc_status_t s : list)
        if (s != DWC_OK) return s;
    return DWC_OK;
}

dwc_status_t make_dropout(double p, unsigned long long seed, unsigned long long offset,
                          const unsigned long long* step, Dropout& d) {
    if (!(p >= 0.0 && p <= 1.0)) return DWC_ERR_INVALID_ARG;
    if (misaligned(step, 8)) return DWC_ERR_ALIGNMENT;
    d.threshold = static_cast<uint32_t>(std::floor(p * 65536.0 + 0.5));
    d.scale = d.threshold < 65536u ? static_cast<float>(65536.0 / (65536.0 - d.threshold)) : 0.f;
    d.k0 = static_cast<uint32_t>(seed);
    d.k1 = static_cast<uint32_t>(seed >> 32);
    d.offset = offset;
    d.step = step;
    return DWC_OK;
}

dwc_status_t map_cuda(cudaError_t err) {
    if (err == cudaSuccess) return DWC_OK;
    (void)cudaGetLastError();  // do not leave the failure to the next launch check
    return DWC_ERR_CUDA;
}

// Whether a tensor's rows start at the same element of a vector of 8 as dense rows from an aligned
// base do (one row: any stride).
bool lines_up(const void* t, int bytes, long long ld, long long rows, int C) {
    return t == nullptr || (!misaligned(t, 8 * static_cast<size_t>(bytes)) && (rows == 1 || (ld - C) % 8 == 0));
}

#define DWC_BY_PAIR(fn, p)                                                                 \
    if ((p).stream_type == kF32) {                                                         \
        if ((p).branch_type == kF32) return fn##_f32(p);                                   \
        return (p).branch_type == kBF16 ? fn##_f32_bf16(p) : fn##_f32_f16(p);              \
    }                                                                                      \
    return (p).stream_type == kBF16 ? fn##_bf16(p) : fn##_f16(p);

cudaError_t fwd_rows(const NormFwd& p) { DWC_BY_PAIR(launch_norm_fwd, p) }
cudaError_t bwd_rows(const NormBwd& p) { DWC_BY_PAIR(launch_norm_bwd, p) }

cudaError_t launch_fwd(const NormFwd& p) {
    const int ws = elem_bytes(p.stream_type), wb = elem_bytes(p.branch_type);
    if (lines_up(p.in, ws, p.ld_in, p.rows, p.C) && lines_up(p.x, wb, p.ld_x, p.rows, p.C) &&
        lines_up(p.z, ws, p.C, p.rows, p.C) && lines_up(p.y, wb, p.C, p.rows, p.C)) {
        const cudaError_t err = fwd_rows(p);
        if (err != cudaErrorNotSupported) return err;
    }
    return launch_norm_fwd_general(p);
}

cudaError_t launch_bwd(const NormBwd& p) {
    const int ws = elem_bytes(p.stream_type), wb = elem_bytes(p.branch_type);
    if (lines_up(p.dy, wb, p.ld_dy, p.rows, p.C) && lines_up(p.dz, ws, p.ld_dz, p.rows, p.C) &&
        lines_up(p.z, ws, p.ld_z, p.rows, p.C) && lines_up(p.d_stream, ws, p.C, p.rows, p.C) &&
        lines_up(p.d_branch, wb, p.C, p.rows, p.C)) {
        const cudaError_t err = bwd_rows(p);
        if (err != cudaErrorNotSupported) return err;
    }
    return launch_norm_bwd_general(p);
}

dwc_status_t norm_fwd(NormFwd& p, dwc_dtype_t stream_type, dwc_dtype_t branch_type, dwc_dtype_t param_dtype) {
    if (!valid_pair(stream_type, branch_type) || !known(param_dtype)) return DWC_ERR_INVALID_ARG;
    if (!(p.eps >= 0.f) || !std::isfinite(p.eps)) return DWC_ERR_INVALID_ARG;
    dwc_status_t st = check_rows(p.rows, p.C);
    if (st != DWC_OK) return st;
    const int ws = elem_bytes(stream_type), wb = elem_bytes(branch_type), wp = elem_bytes(param_dtype);
    const bool add = p.z != nullptr || p.x != nullptr;
    st = first_error({check_tensor(p.in, p.ld_in, p.rows, p.C, ws, false),
                      add ? check_tensor(p.x, p.ld_x, p.rows, p.C, wb, false) : DWC_OK,
                      add ? check_tensor(p.z, p.C, p.rows, p.C, ws, false) : DWC_OK,
                      check_tensor(p.y, p.C, p.rows, p.C, wb, false)});
    if (st != DWC_OK) return st;
    if (misaligned(p.gamma, wp) || misaligned(p.beta, wp) || misaligned(p.mean, 4) || misaligned(p.rstd, 4))
        return DWC_ERR_ALIGNMENT;
    const auto over = [&](const void* out, int type) {
        return first_error({check_in_place(out, type, p.in, p.ld_in, stream_type, p.rows, p.C, p.in_place),
                            check_in_place(out, type, p.x, p.ld_x, branch_type, p.rows, p.C, p.in_place)});
    };
    st = first_error({over(p.y, branch_type), add ? over(p.z, stream_type) : DWC_OK});
    if (st != DWC_OK) return st;
    if (p.rows == 0) return DWC_OK;
    p.stream_type = stream_type;
    p.branch_type = branch_type;
    p.param_type = param_dtype;
    p.status = status_word();
    p.wait_ns = wait_limit_ns();
    return map_cuda(launch_fwd(p));
}

dwc_status_t norm_bwd(NormBwd& p, dwc_dtype_t stream_type, dwc_dtype_t branch_type, dwc_dtype_t param_dtype,
                      void* workspace, size_t workspace_bytes) {
    if (!valid_pair(stream_type, branch_type) || !known(param_dtype)) return DWC_ERR_INVALID_ARG;
    dwc_status_t st = check_rows(p.rows, p.C);
    if (st != DWC_OK) return st;
    const int ws = elem_bytes(stream_type), wb = elem_bytes(branch_type), wp = elem_bytes(param_dtype);
    if (p.rows > 0 && (p.mean == nullptr || p.rstd == nullptr)) return DWC_ERR_INVALID_ARG;
    st = first_error({check_tensor(p.dy, p.ld_dy, p.rows, p.C, wb, false),
                      check_tensor(p.dz, p.ld_dz, p.rows, p.C, ws, true),
                      check_tensor(p.z, p.ld_z, p.rows, p.C, ws, false),
                      check_tensor(p.d_stream, p.C, p.rows, p.C, ws, false),
                      check_tensor(p.d_branch, p.C, p.rows, p.C, wb, true)});
    if (st != DWC_OK) return st;
    if (misaligned(p.gamma, wp) || misaligned(p.mean, 4) || misaligned(p.rstd, 4) || misaligned(p.dgamma, 4) ||
        misaligned(p.dbeta, 4))
        return DWC_ERR_ALIGNMENT;
    const auto over = [&](const void* out, int type) {
        return first_error({check_in_place(out, type, p.dy, p.ld_dy, branch_type, p.rows, p.C, p.in_place),
                            check_in_place(out, type, p.dz, p.ld_dz, stream_type, p.rows, p.C, p.in_place),
                            check_in_place(out, type, p.z, p.ld_z, stream_type, p.rows, p.C, p.in_place)});
    };
    st = first_error({over(p.d_stream, stream_type), over(p.d_branch, branch_type)});
    if (st != DWC_OK) return st;
    const bool params = p.dgamma != nullptr || p.dbeta != nullptr;
    if (p.rows == 0) {
        for (float* d : {p.dgamma, p.dbeta}) {
            if (d == nullptr) continue;
            const cudaError_t err = cudaMemsetAsync(d, 0, static_cast<size_t>(p.C) * sizeof(float), p.stream);
            if (err != cudaSuccess) return map_cuda(err);
        }
        return DWC_OK;
    }
    if (params) {
        if (workspace == nullptr || workspace_bytes < dwc_layer_norm_bwd_workspace_size(p.rows, p.C))
            return DWC_ERR_WORKSPACE;
        if (misaligned(workspace, 16)) return DWC_ERR_ALIGNMENT;
        p.partial = static_cast<float*>(workspace);
    }
    p.stream_type = stream_type;
    p.branch_type = branch_type;
    p.param_type = param_dtype;
    p.status = status_word();
    p.wait_ns = wait_limit_ns();
    return map_cuda(launch_bwd(p));
}

dwc_status_t dropout(const void* x, long long ldx, void* y, long long rows, int C, double p,
                     unsigned long long seed, unsigned long long offset, const unsigned long long* step,
                     dwc_dtype_t dtype, dwc_stream_t stream) {
    if (!known(dtype)) return DWC_ERR_INVALID_ARG;
    DropoutCall c{};
    dwc_status_t st = check_rows(rows, C);
    if (st != DWC_OK) return st;
    const int bytes = elem_bytes(dtype);
    st = first_error({make_dropout(p, seed, offset, step, c.drop), check_tensor(x, ldx, rows, C, bytes, false),
                      check_tensor(y, C, rows, C, bytes, false)});
    if (st != DWC_OK) return st;
    bool in_place = false;
    st = check_in_place(y, dtype, x, ldx, dtype, rows, C, in_place);
    if (st != DWC_OK) return st;
    if (rows == 0) return DWC_OK;
    c.x = x;
    c.y = y;
    c.rows = rows;
    c.ld_x = ldx;
    c.C = C;
    c.type = dtype;
    c.stream = stream;
    if (lines_up(x, bytes, ldx, rows, C) && lines_up(y, bytes, C, rows, C)) {
        const cudaError_t err = launch_dropout_vec(c);
        if (err != cudaErrorNotSupported) return map_cuda(err);
    }
    return map_cuda(launch_dropout_general(c));
}

}  // namespace

extern "C" {

dwc_status_t dwc_layer_norm_fwd(const void* x, long long ldx, const void* gamma, const void* beta,
                                dwc_dtype_t param_dtype, float eps, void* y, float* mean, float* rstd,
                                long long rows, int C, dwc_dtype_t dtype, dwc_dtype_t out_dtype,
                                dwc_stream_t stream) {
    NormFwd p{};
    p.in = x;
    p.ld_in = ldx;
    p.gamma = gamma;
    p.beta = beta;
    p.eps = eps;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    p.rows = rows;
    p.C = C;
    p.stream = stream;
    return norm_fwd(p, dtype, out_dtype, param_dtype);
}

size_t dwc_layer_norm_bwd_workspace_size(long long rows, int C) {
    if (check_rows(rows, C) != DWC_OK || rows == 0) return 0;
    return static_cast<size_t>(norm_bwd_partials(rows, C)) * 2 * C * sizeof(float);
}

dwc_status_t dwc_layer_norm_bwd(const void* dy, long long lddy, const void* x, long long ldx, const float* mean,
                                const float* rstd, const void* gamma, dwc_dtype_t param_dtype, void* dx,
                                float* dgamma, float* dbeta, long long rows, int C, dwc_dtype_t dtype,
                                dwc_dtype_t dy_dtype, void* workspace, size_t workspace_bytes,
                                dwc_stream_t stream) {
    NormBwd p{};
    p.dy = dy;
    p.ld_dy = lddy;
    p.z = x;
    p.ld_z = ldx;
    p.mean = mean;
    p.rstd = rstd;
    p.gamma = gamma;
    p.d_stream = dx;
    p.dgamma = dgamma;
    p.dbeta = dbeta;
    p.rows = rows;
    p.C = C;
    p.stream = stream;
    return norm_bwd(p, dtype, dy_dtype, param_dtype, workspace, workspace_bytes);
}

dwc_status_t dwc_dropout_fwd(const void* x, long long ldx, void* y, long long rows, int C, double p,
                             unsigned long long seed, unsigned long long offset, const unsigned long long* step,
                             dwc_dtype_t dtype, dwc_stream_t stream) {
    return dropout(x, ldx, y, rows, C, p, seed, offset, step, dtype, stream);
}

dwc_status_t dwc_dropout_bwd(const void* dy, long long lddy, void* dx, long long rows, int C, double p,
                             unsigned long long seed, unsigned long long offset, const unsigned long long* step,
                             dwc_dtype_t dtype, dwc_stream_t stream) {
    return dropout(dy, lddy, dx, rows, C, p, seed, offset, step, dtype, stream);
}

dwc_status_t dwc_add_layer_norm_fwd(const void* x, long long ldx, const void* res, long long ldres, double p,
                                    unsigned long long seed, unsigned long long offset,
                                    const unsigned long long* step, const void* gamma, const void* beta,
                                    dwc_dtype_t param_dtype, float eps, void* z, void* y, float* mean,
                                    float* rstd, long long rows, int C, dwc_dtype_t dtype,
                                    dwc_dtype_t res_dtype, dwc_stream_t stream) {
    NormFwd f{};
    const dwc_status_t st = make_dropout(p, seed, offset, step, f.drop);
    if (st != DWC_OK) return st;
    if (rows > 0 && (x == nullptr || z == nullptr)) return DWC_ERR_INVALID_ARG;
    f.in = res;
    f.ld_in = ldres;
    f.x = x;
    f.ld_x = ldx;
    f.gamma = gamma;
    f.beta = beta;
    f.eps = eps;
    f.z = z;
    f.y = y;
    f.mean = mean;
    f.rstd = rstd;
    f.rows = rows;
    f.C = C;
    f.stream = stream;
    return norm_fwd(f, res_dtype, dtype, param_dtype);
}

dwc_status_t dwc_add_layer_norm_bwd(const void* dy, long long lddy, const void* dz, long long lddz, const void* z,
                                    long long ldz, const float* mean, const float* rstd, const void* gamma,
                                    dwc_dtype_t param_dtype, double p, unsigned long long seed,
                                    unsigned long long offset, const unsigned long long* step, void* dx,
                                    void* dres, float* dgamma, float* dbeta, long long rows, int C,
                                    dwc_dtype_t dtype, dwc_dtype_t res_dtype, void* workspace,
                                    size_t workspace_bytes, dwc_stream_t stream) {
    NormBwd b{};
    const dwc_status_t st = make_dropout(p, seed, offset, step, b.drop);
    if (st != DWC_OK) return st;
    // without dropout and conversion dx would be dres again, and only then may it be left out
    if (rows > 0 && dx == nullptr && (b.drop.threshold != 0 || dtype != res_dtype)) return DWC_ERR_INVALID_ARG;
    b.dy = dy;
    b.ld_dy = lddy;
    b.dz = dz;
    b.ld_dz = lddz;
    b.z = z;
    b.ld_z = ldz;
    b.mean = mean;
    b.rstd = rstd;
    b.gamma = gamma;
    b.d_stream = dres;
    b.d_branch = dx;
    b.dgamma = dgamma;
    b.dbeta = dbeta;
    b.rows = rows;
    b.C = C;
    b.stream = stream;
    return norm_bwd(b, res_dtype, dtype, param_dtype, workspace, workspace_bytes);
}

}  // extern "C"
