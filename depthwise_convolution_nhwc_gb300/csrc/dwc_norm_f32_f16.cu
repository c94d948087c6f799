// dwc_norm_f32_f16.cu -- layer norm rows kernels for an fp32 stream with fp16 branches.
#include "dwc_norm_rows.cuh"

namespace dwc {

cudaError_t launch_norm_fwd_f32_f16(const NormFwd& p) {
    return p.x != nullptr ? norm::fwd_rows<float, __half, true>(p) : norm::fwd_rows<float, __half, false>(p);
}
cudaError_t launch_norm_bwd_f32_f16(const NormBwd& p) {
    const bool add = p.dz != nullptr || p.d_branch != nullptr;
    return add ? norm::bwd_rows<float, __half, true>(p) : norm::bwd_rows<float, __half, false>(p);
}

}  // namespace dwc
