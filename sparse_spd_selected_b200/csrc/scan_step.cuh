// The selective scan for single tokens: one row per sequence over a cache of
// states [slots, d, n].  Bounded by memory, the states read and written once:
// a thread takes four neighbouring states of one channel, the LN lanes of a
// channel add their parts of y.
#pragma once

#include "conv.cuh"
#include "scan.cuh"

namespace selinv {
namespace {

constexpr int STEP_THREADS = 256;

template <class T, int LN>
__global__ void __launch_bounds__(STEP_THREADS) scan_step_kernel(const __grid_constant__ ScanStepArgs p)
{
    using C = typename Elem<T>::C;
    constexpr int CH = STEP_THREADS / LN;
    const int64_t blocks = (p.d + CH - 1) / CH, r = blockIdx.x / blocks;
    const int64_t c = (blockIdx.x % blocks) * CH + threadIdx.x / LN;
    const int64_t slot = step_slot(p.index, p.info, r, p.slots, blockIdx.x % blocks == 0);
    const int lane = threadIdx.x % 32, n0 = (threadIdx.x % LN) * 4, n = p.n;
    const bool in = c < p.d;
    T *y = static_cast<T *>(p.y) + r * p.y_row + c;
    if (slot < 0) {
        if (in && threadIdx.x % LN == 0) *y = Elem<T>::down((C)0);
        return;
    }
    C v[1] = {0}, x = 0;
    if (in) {
        const int64_t at = (slot * p.d + c) * n + n0, g = c / (p.d / p.groups);
        const C *h = static_cast<const C *>(p.cache) + at, *A = static_cast<const C *>(p.A) + c * n + n0;
        C *out = static_cast<C *>(p.cache_out) + at;
        const T *B = static_cast<const T *>(p.B) + r * p.B_row + g * p.B_group + n0;
        const T *Cc = static_cast<const T *>(p.C) + r * p.C_row + g * p.C_group + n0;
        C hs[4], as[4];
        const bool wide = n % 4 == 0 && sizeof(C) == 4 &&
                          ((uintptr_t)p.cache | (uintptr_t)p.cache_out | (uintptr_t)p.A) % 16 == 0;
        if (wide && n0 < n) {
            get<4>(h, hs);
            get<4>(A, as);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                hs[j] = n0 + j < n ? h[j] : (C)0;
                as[j] = n0 + j < n ? A[j] : (C)0;
            }
        }
        x = Elem<T>::up(static_cast<const T *>(p.x)[r * p.x_row + c]);
        C dt = Elem<T>::up(static_cast<const T *>(p.dt)[r * p.dt_row + c]);
        if (p.dt_bias) dt += static_cast<const C *>(p.dt_bias)[c];
        if (p.softplus) dt = softplus_(dt);
        const C u = dt * x, d2 = dt * log2e<C>();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + j < n) {
                hs[j] = exp2_(d2 * as[j]) * hs[j] + u * Elem<T>::up(B[j]);
                v[0] += Elem<T>::up(Cc[j]) * hs[j];
            }
        if (wide && n0 < n) {
            put<4>(out, hs);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < n) out[j] = hs[j];
        }
    }
    scatter_sum<1, 1, LN>(v, lane);
    if (in && threadIdx.x % LN == 0) {
        C t = v[0];
        if (p.D) t += static_cast<const C *>(p.D)[c] * x;
        if (p.z) {
            const C z = Elem<T>::up(static_cast<const T *>(p.z)[r * p.z_row + c]);
            t *= z * sigmoid_(z);
        }
        *y = Elem<T>::down(t);
    }
}

template <class T, int LN> cudaError_t scan_step_run(const ScanStepArgs &p, cudaStream_t s)
{
    constexpr int CH = STEP_THREADS / LN;
    const int64_t blocks = (p.d + CH - 1) / CH * p.batch;
    scan_step_kernel<T, LN><<<(unsigned)blocks, STEP_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
