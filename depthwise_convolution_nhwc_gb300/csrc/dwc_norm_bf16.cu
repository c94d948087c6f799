// dwc_norm_bf16.cu -- layer norm rows kernels for bf16.
#include "dwc_norm_rows.cuh"

namespace dwc {

cudaError_t launch_norm_fwd_bf16(const NormFwd& p) {
    return p.x != nullptr ? norm::fwd_rows<__nv_bfloat16, __nv_bfloat16, true>(p) : norm::fwd_rows<__nv_bfloat16, __nv_bfloat16, false>(p);
}
cudaError_t launch_norm_bwd_bf16(const NormBwd& p) {
    const bool add = p.dz != nullptr || p.d_branch != nullptr;
    return add ? norm::bwd_rows<__nv_bfloat16, __nv_bfloat16, true>(p) : norm::bwd_rows<__nv_bfloat16, __nv_bfloat16, false>(p);
}

}  // namespace dwc
