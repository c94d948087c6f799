// dwc_norm_f16.cu -- layer norm rows kernels for fp16.
#include "dwc_norm_rows.cuh"

namespace dwc {

cudaError_t launch_norm_fwd_f16(const NormFwd& p) {
    return p.x != nullptr ? norm::fwd_rows<__half, __half, true>(p) : norm::fwd_rows<__half, __half, false>(p);
}
cudaError_t launch_norm_bwd_f16(const NormBwd& p) {
    const bool add = p.dz != nullptr || p.d_branch != nullptr;
    return add ? norm::bwd_rows<__half, __half, true>(p) : norm::bwd_rows<__half, __half, false>(p);
}

}  // namespace dwc
