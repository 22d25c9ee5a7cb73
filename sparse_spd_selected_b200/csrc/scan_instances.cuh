// The scan's kernels for one element type (included once per type).
#pragma once

#include "scan_backward.cuh"
#include "scan_forward.cuh"
#include "scan_step.cuh"
#include "sequence.h"

namespace selinv {

static_assert(SCAN_R == SCAN_KEEP_ROWS && SCAN_WARPS == SCAN_BLOCK_TILES, "the host sizes buffers by these");

namespace {

template <class T, int NP> struct Tiles {
    using Narrow = ScanTile<T, 2, 2, NP / 2>;
    using Wide = std::conditional_t<sizeof(T) == 8, Narrow, ScanTile<T, 4, 4, NP / 4>>;
};

// Calls f with the tile type for n states; the backward keeps a tile's states in shared memory, where not every wide
// tile fits.
template <class T, bool BACKWARD, class F> auto with_tile(int n, bool narrow, F f)
{
    auto pick = [&](auto t) {
        using P = decltype(t);
        if constexpr (!std::is_same<typename P::Wide, typename P::Narrow>::value &&
                      (!BACKWARD || sizeof(ScanBwdBlock<typename P::Wide>) <= 227 * 1024))
            if (!narrow) return f(typename P::Wide());
        return f(typename P::Narrow());
    };
    if (n <= 4) return pick(Tiles<T, 4>());
    if (n <= 8) return pick(Tiles<T, 8>());
    if (n <= 16) return pick(Tiles<T, 16>());
    if (n <= 32) return pick(Tiles<T, 32>());
    return pick(Tiles<T, 64>());
}

}  // namespace

template <class T> int scan_tile_channels(int n, bool narrow, bool backward)
{
    const auto cw = [](auto k) { return decltype(k)::CW; };
    return backward ? with_tile<T, true>(n, narrow, cw) : with_tile<T, false>(n, narrow, cw);
}
template <class T> cudaError_t scan_launch(const ScanArgs &p, bool narrow, cudaStream_t s)
{
    return with_tile<T, false>(p.n, narrow, [&](auto k) { return scan_run<decltype(k)>(p, s); });
}
template <class T> cudaError_t scan_backward_launch(const ScanArgs &p, const ScanGrads &o, bool narrow, cudaStream_t s)
{
    return with_tile<T, true>(p.n, narrow, [&](auto k) { return scan_backward_run<decltype(k)>(p, o, s); });
}
template <class T> cudaError_t scan_step_launch(const ScanStepArgs &p, cudaStream_t s)
{
    if (p.n <= 4) return scan_step_run<T, 1>(p, s);
    if (p.n <= 8) return scan_step_run<T, 2>(p, s);
    if (p.n <= 16) return scan_step_run<T, 4>(p, s);
    if (p.n <= 32) return scan_step_run<T, 8>(p, s);
    return scan_step_run<T, 16>(p, s);
}

#define SELINV_SCAN_INSTANCES(T)                                                            \
    template int scan_tile_channels<T>(int, bool, bool);                                       \
    template cudaError_t scan_launch<T>(const ScanArgs &, bool, cudaStream_t);              \
    template cudaError_t scan_backward_launch<T>(const ScanArgs &, const ScanGrads &, bool, cudaStream_t); \
    template cudaError_t scan_step_launch<T>(const ScanStepArgs &, cudaStream_t);

}  // namespace selinv
