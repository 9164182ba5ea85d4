// The selective scan's kernels for bf16 tensors (ssm_scan.h).
#include "ssm_scan.h"

namespace gdn {
hipError_t launch_ssm_scan_bf16(const SsmScans& a, int count, int dk, int dv, int mode, hipStream_t s) {
  return run_ssm_scan_dims<bf16>(a, count, dk, dv, mode, s);
}
}  // namespace gdn
