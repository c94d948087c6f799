// dwc_scan_bf16.cu -- selective scan kernels for bf16.
#include "dwc_scan.cuh"

namespace dwc {

cudaError_t launch_scan_fwd_bf16(const Scan& p) { return scan::fwd<__nv_bfloat16>(p); }
cudaError_t launch_scan_bwd_bf16(const Scan& p) { return scan::bwd<__nv_bfloat16>(p); }

}  // namespace dwc
