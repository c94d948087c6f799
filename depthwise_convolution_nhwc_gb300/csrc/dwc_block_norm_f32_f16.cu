// dwc_block_norm_f32_f16.cu -- block norm rows kernels for an fp32 stream with fp16 branches.
#include "dwc_block_norm_rows.cuh"

namespace dwc {

cudaError_t launch_block_norm_fwd_f32_f16(const BlockNorm& p) { return block_norm::fwd_rows<float, __half>(p); }
cudaError_t launch_block_norm_bwd_f32_f16(const BlockNorm& p) { return block_norm::bwd_rows<float, __half>(p); }

}  // namespace dwc
