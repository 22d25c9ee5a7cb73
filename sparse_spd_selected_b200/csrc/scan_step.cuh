// The selective scan for single tokens: one row per sequence over a cache of
// states [slots, d, n].  Bounded by memory, the states read and written once.
// Each lane has a channel of its own for what a channel has once (step, gate,
// y); for the states LN neighbouring lanes take their LN channels one after
// another, four states of each a lane, so that the loads and stores of 16
// bytes cover whole sectors.  192 rows of 4096 x 16: 28 us for 107 MB, 3.8 TB/s
// (0.58 of a plain copy's rate); every row's blocks read A again, as many bytes
// as the states, from L2.  Held to 64 registers for eight blocks per SM it took
// 30.  One row of 2048 x 16: 4.7 us, a launch and two waits for memory.
#pragma once

#include "conv.cuh"
#include "scan.cuh"

namespace selinv {
namespace {

constexpr int STEP_THREADS = 128;

template <class T, int LN>
__global__ void __launch_bounds__(STEP_THREADS) scan_step_kernel(const __grid_constant__ ScanStepArgs p)
{
    using C = typename Elem<T>::C;
    const unsigned blocks = (unsigned)((p.d + STEP_THREADS - 1) / STEP_THREADS), row = blockIdx.x / blocks;
    const int bi = (int)(blockIdx.x - row * blocks);
    const int64_t r = row;
    const int64_t slot = step_slot(p.index, r, p.slots);
    const int lane = threadIdx.x % 32, nl = threadIdx.x % LN, n0 = nl * 4, n = p.n, d = (int)p.d;
    const int c = bi * STEP_THREADS + threadIdx.x, first = c - nl;      // this lane's channel, and its lanes' first
    const bool in = c < d;
    const bool wide = n % 4 == 0 && sizeof(C) == 4 &&
                      ((uintptr_t)p.cache | (uintptr_t)p.cache_out | (uintptr_t)p.A) % 16 == 0;
    constexpr int U = LN < 4 ? LN : 4;          // channels whose loads are on their way together
    C h[U][4], a[U][4];
    const int64_t at = (slot * d + first) * n + n0;     // the lane's states of its first channel
    const C *const hs0 = static_cast<const C *>(p.cache) + at, *const as0 = static_cast<const C *>(p.A) + ((int64_t)first * n + n0);
    C *const out0 = static_cast<C *>(p.cache_out) + at;
    const auto load = [&](int u0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = first + u0 + u;
            const C *hs = hs0 + (u0 + u) * n, *as = as0 + (u0 + u) * n;
            const bool have = slot >= 0 && ch < d && n0 < n;
            if (have && wide) {
                get<4>(hs, h[u]);
                get<4>(as, a[u]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[u][j] = have && n0 + j < n ? hs[j] : (C)0;
                    a[u][j] = have && n0 + j < n ? as[j] : (C)0;
                }
            }
        }
    };
    load(0);
    C x = 0, dt = 0, z = 0, skip = 0;
    if (in) {
        x = Elem<T>::up(static_cast<const T *>(p.x)[r * p.x_row + c]);
        dt = Elem<T>::up(static_cast<const T *>(p.dt)[r * p.dt_row + c]);
        if (p.dt_bias) dt += static_cast<const C *>(p.dt_bias)[c];
        if (p.z) z = Elem<T>::up(static_cast<const T *>(p.z)[r * p.z_row + c]);
        if (p.D) skip = static_cast<const C *>(p.D)[c];
    }
    const bool ours = step_first(p.index, p.info, r, slot, bi == 0);
    T *y = static_cast<T *>(p.y) + r * p.y_row + c;
    if (!ours) {
        if (in) *y = Elem<T>::down((C)0);
        return;
    }
    const int per = p.groups == 1 ? d : d / p.groups;
    C b[4], cc[4], v[LN];
    int group = -1;
    if (p.softplus) dt = softplus_of<T>(dt);
    const C ux = dt * x, d2 = dt * log2e<C>();
#pragma unroll
    for (int u0 = 0; u0 < LN; u0 += U) {
        if (u0) load(u0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int ch = first + u0 + u, from = lane - nl + u0 + u;
            const int g = ch >= d ? group : p.groups == 1 ? 0 : ch / per;
            if (g != group) {       // once in a call with one group
                group = g;
                const T *B = static_cast<const T *>(p.B) + r * p.B_row + g * p.B_group + n0;
                const T *Cc = static_cast<const T *>(p.C) + r * p.C_row + g * p.C_group + n0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b[j] = n0 + j < n ? Elem<T>::up(B[j]) : (C)0;
                    cc[j] = n0 + j < n ? Elem<T>::up(Cc[j]) : (C)0;
                }
            }
            const C e = LN > 1 ? __shfl_sync(FULL_MASK, d2, from) : d2, w = LN > 1 ? __shfl_sync(FULL_MASK, ux, from) : ux;
            v[u0 + u] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < n) {
                    h[u][j] = exp2_(e * a[u][j]) * h[u][j] + w * b[j];
                    v[u0 + u] += cc[j] * h[u][j];
                }
            if (ch < d && n0 < n) {
                C *out = out0 + (u0 + u) * n;
                if (wide) {
                    put<4>(out, h[u]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n0 + j < n) out[j] = h[u][j];
                }
            }
        }
    }
    scatter_sum<LN, 1, LN>(v, lane);        // each lane ends with its own channel's sum
    if (in) {
        C t = v[0] + skip * x;
        if (p.z) t *= z * sigmoid_(z);
        *y = Elem<T>::down(t);
    }
}

template <class T, int LN> cudaError_t scan_step_run(const ScanStepArgs &p, cudaStream_t s)
{
    const int64_t blocks = (p.d + STEP_THREADS - 1) / STEP_THREADS * p.batch;
    scan_step_kernel<T, LN><<<(unsigned)blocks, STEP_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
