// The selective scan's kernels for f32 sequences.
#include "scan_instances.cuh"

namespace selinv {
SELINV_SCAN_INSTANCES(float)
}  // namespace selinv
