// The scan's kernels for one element type (included once per type).
#pragma once

#include "scan_backward.cuh"
#include "scan_forward.cuh"
#include "scan_step.cuh"
#include "sequence.h"

namespace selinv {

static_assert(SCAN_R == SCAN_KEEP_ROWS && SCAN_WARPS == SCAN_BLOCK_TILES, "the host sizes buffers by these");

namespace {

// Calls f with the number of states rounded up to one that kernels exist for.
template <class F> auto with_states(int n, F f)
{
    if (n <= 4) return f(std::integral_constant<int, 4>());
    if (n <= 8) return f(std::integral_constant<int, 8>());
    if (n <= 16) return f(std::integral_constant<int, 16>());
    if (n <= 32) return f(std::integral_constant<int, 32>());
    return f(std::integral_constant<int, 64>());
}
}  // namespace

template <class T> int scan_backward_channels(int n)
{
    return with_states(n, [](auto np) { return ScanBwdTile<T, np.value>::CW; });
}
template <class T> int scan_backward_blocks(int n)
{
    return with_states(n, [](auto np) { return scan_bwd_blocks<ScanBwdTile<T, np.value>>; });
}
template <class T> cudaError_t scan_launch(const ScanArgs &p, int lanes, cudaStream_t s)
{
    return with_states(p.n, [&](auto np) {
        return with_lanes<T, np.value>(lanes, [&](auto k) { return scan_run<decltype(k)>(p, s); });
    });
}
template <class T> cudaError_t scan_backward_launch(const ScanArgs &p, const ScanGrads &o, cudaStream_t s)
{
    return with_states(p.n, [&](auto np) { return scan_backward_run<T, np.value>(p, o, s); });
}
template <class T> cudaError_t scan_step_launch(const ScanStepArgs &p, cudaStream_t s)
{
    if (p.n <= 4) return scan_step_run<T, 1>(p, s);
    if (p.n <= 8) return scan_step_run<T, 2>(p, s);
    if (p.n <= 16) return scan_step_run<T, 4>(p, s);
    if (p.n <= 32) return scan_step_run<T, 8>(p, s);
    return scan_step_run<T, 16>(p, s);
}

#define SELINV_SCAN_INSTANCES(T)                                                                   \
    template int scan_backward_channels<T>(int);                                                   \
    template int scan_backward_blocks<T>(int);                                                     \
    template cudaError_t scan_launch<T>(const ScanArgs &, int, cudaStream_t);                      \
    template cudaError_t scan_backward_launch<T>(const ScanArgs &, const ScanGrads &, cudaStream_t); \
    template cudaError_t scan_step_launch<T>(const ScanStepArgs &, cudaStream_t);

}  // namespace selinv
