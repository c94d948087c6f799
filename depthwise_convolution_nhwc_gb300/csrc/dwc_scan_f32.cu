// dwc_scan_f32.cu -- selective scan kernels for fp32.
#include "dwc_scan.cuh"

namespace dwc {

cudaError_t launch_scan_fwd_f32(const Scan& p) { return scan::fwd<float>(p); }
cudaError_t launch_scan_bwd_f32(const Scan& p) { return scan::bwd<float>(p); }

}  // namespace dwc
