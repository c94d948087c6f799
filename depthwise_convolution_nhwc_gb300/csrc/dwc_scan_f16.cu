// dwc_scan_f16.cu -- selective scan kernels for fp16.
#include "dwc_scan.cuh"

namespace dwc {

cudaError_t launch_scan_fwd_f16(const Scan& p) { return scan::fwd<__half>(p); }
cudaError_t launch_scan_bwd_f16(const Scan& p) { return scan::bwd<__half>(p); }

}  // namespace dwc
