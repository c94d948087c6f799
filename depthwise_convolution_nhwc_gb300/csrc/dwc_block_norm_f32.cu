// dwc_block_norm_f32.cu -- block norm rows kernels for fp32.
#include "dwc_block_norm_rows.cuh"

namespace dwc {

cudaError_t launch_block_norm_fwd_f32(const BlockNorm& p) { return block_norm::fwd_rows<float, float>(p); }
cudaError_t launch_block_norm_bwd_f32(const BlockNorm& p) { return block_norm::bwd_rows<float, float>(p); }

}  // namespace dwc
