// Launchers of the sequence operators, one set per element type.
#pragma once

#include "sequence.cuh"

namespace selinv {

// States are padded to 4, 8, 16, 32 or 64.  In the forward 1, 2 or 4 lanes share a channel, none with more than 16
// states or fewer than 4; a warp has 32 / lanes channels.
constexpr int scan_least_lanes(int n) { return n <= 16 ? 1 : n <= 32 ? 2 : 4; }
constexpr int scan_most_lanes(int n) { return n <= 4 ? 1 : n <= 8 ? 2 : 4; }
template <class T> int scan_backward_channels(int n);
template <class T> int scan_backward_blocks(int n);     // resident per SM
template <class T> cudaError_t scan_launch(const ScanArgs &p, int lanes, cudaStream_t s);
template <class T> cudaError_t scan_backward_launch(const ScanArgs &p, const ScanGrads &o, cudaStream_t s);
template <class T> cudaError_t scan_step_launch(const ScanStepArgs &p, cudaStream_t s);
template <class T> cudaError_t conv_launch(const ConvArgs &p, cudaStream_t s);
template <class T> cudaError_t conv_backward_launch(const ConvArgs &p, cudaStream_t s);
template <class T> cudaError_t conv_step_launch(const ConvStepArgs &p, cudaStream_t s);

constexpr int SCAN_MAX_N = 64, CONV_MIN_K = 2, CONV_MAX_K = 8;
constexpr int scan_padded(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : n <= 16 ? 16 : n <= 32 ? 32 : 64; }
constexpr int SCAN_KEEP_ROWS = 16;      // rows between the states kept for the backward
constexpr int SCAN_BLOCK_TILES = 4;     // warp tiles of a block

}  // namespace selinv
