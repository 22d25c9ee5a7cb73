// The selective scan's kernels for f64 sequences.
#include "scan_instances.cuh"

namespace selinv {
SELINV_SCAN_INSTANCES(double)
}  // namespace selinv
