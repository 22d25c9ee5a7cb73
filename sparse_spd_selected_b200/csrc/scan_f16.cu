// The selective scan's kernels for f16 sequences.
#include "scan_instances.cuh"

namespace selinv {
SELINV_SCAN_INSTANCES(__half)
}  // namespace selinv
