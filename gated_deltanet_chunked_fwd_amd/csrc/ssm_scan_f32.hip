// The selective scan's kernels for fp32 tensors (ssm_scan.h).
#include "ssm_scan.h"

namespace gdn {
hipError_t launch_ssm_scan_f32(const SsmScans& a, int count, int dk, int dv, int mode, hipStream_t s) {
  return run_ssm_scan_dims<float>(a, count, dk, dv, mode, s);
}
}  // namespace gdn
