// The scan's kernels for one element type (included once per type).
#pragma once

#include "scan_backward.cuh"
#include "scan_forward.cuh"
#include "scan_step.cuh"
#include "sequence.h"

namespace selinv {

static_assert(SCAN_R == SCAN_KEEP_ROWS && SCAN_WARPS == SCAN_BLOCK_TILES, "the host sizes buffers by these");

namespace {

// The tile for n states: 4 channels x 4, 2 or 1 states per thread (float64: 2 x 2).  The backward takes the first.
template <class T, int NP, int NARROW> struct TileOf {
    static constexpr int TN = NARROW == 0 ? 4 : NARROW == 1 || NP == 64 ? 2 : 1;
    using K = std::conditional_t<sizeof(T) == 8, ScanTile<T, 2, 2, NP>, ScanTile<T, 16 / sizeof(typename Elem<T>::C), TN, NP>>;
};
template <class T, int NP, class F> auto with_width_of(int narrow, F f)
{
    if (narrow == 0) return f(typename TileOf<T, NP, 0>::K());
    if (narrow == 1) return f(typename TileOf<T, NP, 1>::K());
    return f(typename TileOf<T, NP, 2>::K());
}
// Calls f with the tile type.
template <class T, class F> auto with_tile(int n, int narrow, F f)
{
    if (n <= 4) return with_width_of<T, 4>(narrow, f);
    if (n <= 8) return with_width_of<T, 8>(narrow, f);
    if (n <= 16) return with_width_of<T, 16>(narrow, f);
    if (n <= 32) return with_width_of<T, 32>(narrow, f);
    return with_width_of<T, 64>(narrow, f);
}

}  // namespace

template <class T> int scan_tile_channels(int n, int narrow)
{
    return with_tile<T>(n, narrow, [](auto k) { return decltype(k)::CW; });
}
template <class T> cudaError_t scan_launch(const ScanArgs &p, int narrow, cudaStream_t s)
{
    return with_tile<T>(p.n, narrow, [&](auto k) { return scan_run<decltype(k)>(p, s); });
}
template <class T> cudaError_t scan_backward_launch(const ScanArgs &p, const ScanGrads &o, cudaStream_t s)
{
    if (p.n <= 4) return scan_backward_run<typename TileOf<T, 4, 0>::K>(p, o, s);
    if (p.n <= 8) return scan_backward_run<typename TileOf<T, 8, 0>::K>(p, o, s);
    if (p.n <= 16) return scan_backward_run<typename TileOf<T, 16, 0>::K>(p, o, s);
    if (p.n <= 32) return scan_backward_run<typename TileOf<T, 32, 0>::K>(p, o, s);
    return scan_backward_run<typename TileOf<T, 64, 0>::K>(p, o, s);
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
    template int scan_tile_channels<T>(int, int);                                                  \
    template cudaError_t scan_launch<T>(const ScanArgs &, int, cudaStream_t);                      \
    template cudaError_t scan_backward_launch<T>(const ScanArgs &, const ScanGrads &, cudaStream_t); \
    template cudaError_t scan_step_launch<T>(const ScanStepArgs &, cudaStream_t);

}  // namespace selinv
