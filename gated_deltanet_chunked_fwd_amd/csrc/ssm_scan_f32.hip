// The selective scan's kernels for fp32 tensors (ssm_scan.h).
#include "ssm_scan.h"

namespace gdn {
hipError_t launch_ssm_scan_f32(const SsmScans& a, int count, int dk, int dv, bool state_pass, hipStream_t s) {
  return run_ssm_scan_dims<float>(a, count, dk, dv, state_pass, s);
}
}  // namespace gdn
