// dwc_norm_f32.cu -- layer norm rows kernels for fp32.
#include "dwc_norm_rows.cuh"

namespace dwc {

cudaError_t launch_norm_fwd_f32(const NormFwd& p) {
    return p.x != nullptr ? norm::fwd_rows<float, float, true>(p) : norm::fwd_rows<float, float, false>(p);
}
cudaError_t launch_norm_bwd_f32(const NormBwd& p) {
    const bool add = p.dz != nullptr || p.d_branch != nullptr;
    return add ? norm::bwd_rows<float, float, true>(p) : norm::bwd_rows<float, float, false>(p);
}

}  // namespace dwc
