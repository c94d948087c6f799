// dwc_block_norm_bf16.cu -- block norm rows kernels for bf16.
#include "dwc_block_norm_rows.cuh"

namespace dwc {

cudaError_t launch_block_norm_fwd_bf16(const BlockNorm& p) { return block_norm::fwd_rows<__nv_bfloat16, __nv_bfloat16>(p); }
cudaError_t launch_block_norm_bwd_bf16(const BlockNorm& p) { return block_norm::bwd_rows<__nv_bfloat16, __nv_bfloat16>(p); }

}  // namespace dwc
