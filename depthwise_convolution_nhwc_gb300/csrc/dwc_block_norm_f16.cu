// dwc_block_norm_f16.cu -- block norm rows kernels for fp16.
#include "dwc_block_norm_rows.cuh"

namespace dwc {

cudaError_t launch_block_norm_fwd_f16(const BlockNorm& p) { return block_norm::fwd_rows<__half, __half>(p); }
cudaError_t launch_block_norm_bwd_f16(const BlockNorm& p) { return block_norm::bwd_rows<__half, __half>(p); }

}  // namespace dwc
