// The selective scan's kernels for bf16 sequences.
#include "scan_instances.cuh"

namespace selinv {
SELINV_SCAN_INSTANCES(__nv_bfloat16)
}  // namespace selinv
