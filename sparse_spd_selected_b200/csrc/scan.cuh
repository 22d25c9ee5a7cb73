// The selective scan along chains (sm_100a):
//   dt'_t = softplus(dt_t + dt_bias)   (or without the softplus)
//   h_t   = exp(dt'_t A) h_{t-1} + dt'_t x_t B_t      [d, n] states in 32 bits (64 for float64)
//   y_t   = (sum_n C_t h_t + D x_t) silu(z_t)
// i.e. the solve of the block lower-bidiagonal system with M_tt = I and
// M_{t,t-1} = -diag(exp(dt'_t A)), read out by C.
#pragma once

#include "sequence.cuh"

namespace selinv {
namespace {

// Rows staged at a time, and the spacing of the states kept for the backward pass.
constexpr int SCAN_R = 16;
constexpr int SCAN_WARPS = 4;

// A warp's tile: TD channels x TN states in each thread, LN lanes along the states.
template <class T_, int TD_, int TN_, int LN_> struct ScanTile {
    using T = T_;
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    static constexpr int TD = TD_, TN = TN_, LN = LN_, LD = 32 / LN, CW = LD * TD, NP = LN * TN, TP = TD / 2;
    // channels a lane converts at a time, and lanes' shares of a staged tile
    static constexpr int E = (16 / (int)sizeof(T) < CW) ? 16 / (int)sizeof(T) : CW;
    static constexpr int VECS = SCAN_R * CW / E, PER = (VECS + 31) / 32;
    // elements of B and C a lane converts at a time
    static constexpr int EB = sizeof(T) == 8 ? 2 : 4, BVECS = SCAN_R * NP / EB, BPER = (BVECS + 31) / 32;
    // row pitch of the staged arrays: neighbouring rows start 16 bytes further round the banks (and on 16 bytes)
    static constexpr int PITCH = CW + (CW >= 4 ? 4 : 2);
    static_assert(PITCH * sizeof(C) % 16 == 0, "vectors of 16 bytes in every staged row");
    static_assert(CW % E == 0 && 32 % (CW / E) == 0, "a lane keeps its channels from row to row");
};

// Where a warp works: line and rows, channel group and channels.
struct ScanPlace {
    int64_t line, r0, r1;
    int seg, group, c0, nch;     // c0: first channel (of all d); nch <= CW of them
};

template <class C> struct ScanState {
    const C *in;        // initial states [sequences, d, n] or null
    C *out;             // final states or null
};

// One tile of rows of a 16-bit, 32-bit or 64-bit array [lines, rows, channels], as words in registers.
template <class K, int PER, int E, int PERROW> struct ScanLoad {
    using T = typename K::T;
    Pack<T, E> v[PER];
    // row r0 + vec / PERROW, elements (vec % PERROW) * E on; `n` of them exist, rows up to r1
    SELINV_DEVINL void load(const T *p, int64_t row_stride, int64_t r0, int64_t r1, int n, bool wide, int lane)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int vec = lane + 32 * i, row = vec / PERROW, e = (vec % PERROW) * E;
            v[i].clear();
            if (row < SCAN_R && r0 + row < r1) v[i].load(p + (r0 + row) * row_stride + e, n - e, wide);
        }
    }
};

// Small vectors in shared memory.
template <int N> SELINV_DEVINL void put(float *p, const float *v)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) *reinterpret_cast<float2 *>(p + i) = make_float2(v[i], v[i + 1]);
    }
}
template <int N> SELINV_DEVINL void put(double *p, const double *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<double2 *>(p + i) = make_double2(v[i], v[i + 1]);
}
template <int N> SELINV_DEVINL void get(const float *p, float *v)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + i);
            v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 q = *reinterpret_cast<const float2 *>(p + i);
            v[i] = q.x, v[i + 1] = q.y;
        }
    }
}
template <int N> SELINV_DEVINL void get(const double *p, double *v)
{
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const double2 q = *reinterpret_cast<const double2 *>(p + i);
        v[i] = q.x, v[i + 1] = q.y;
    }
}
template <int N> SELINV_DEVINL void get(const float *p, float2 *v)
{
    float t[2 * N];
    get<2 * N>(p, t);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = make_float2(t[2 * i], t[2 * i + 1]);
}
template <int N> SELINV_DEVINL void get(const double *p, double2 *v)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const double2 *>(p + 2 * i);
}

// The thread's TD x TN part of a [d, n] array (p: its first channel of the warp); what lies outside is `fill`.
template <class K> SELINV_DEVINL void load_part(const typename K::C *p, int n, int nch, int lane, typename K::V (*v)[K::TN],
                                                typename K::C fill)
{
    const int d0 = (lane / K::LN) * K::TD, n0 = (lane % K::LN) * K::TN;
#pragma unroll
    for (int q = 0; q < K::TP; ++q)
#pragma unroll
        for (int j = 0; j < K::TN; ++j) {
            const bool in = n0 + j < n;
            v[q][j].x = in && d0 + 2 * q < nch ? p[(int64_t)(d0 + 2 * q) * n + n0 + j] : fill;
            v[q][j].y = in && d0 + 2 * q + 1 < nch ? p[(int64_t)(d0 + 2 * q + 1) * n + n0 + j] : fill;
        }
}
template <class K> SELINV_DEVINL void store_part(typename K::C *p, int n, int nch, int lane, typename K::V (*v)[K::TN])
{
    const int d0 = (lane / K::LN) * K::TD, n0 = (lane % K::LN) * K::TN;
#pragma unroll
    for (int q = 0; q < K::TP; ++q)
#pragma unroll
        for (int j = 0; j < K::TN; ++j) {
            if (n0 + j >= n) continue;
            if (d0 + 2 * q < nch) p[(int64_t)(d0 + 2 * q) * n + n0 + j] = v[q][j].x;
            if (d0 + 2 * q + 1 < nch) p[(int64_t)(d0 + 2 * q + 1) * n + n0 + j] = v[q][j].y;
        }
}

template <class K> SELINV_DEVINL bool scan_place(const ScanArgs &p, int warp, ScanPlace &w)
{
    const int per = (int)(p.d / p.groups), tiles = (per + K::CW - 1) / K::CW;
    const int blocks = (tiles + SCAN_WARPS - 1) / SCAN_WARPS;
    w.line = blockIdx.x / p.segs;
    w.seg = (int)(blockIdx.x % p.segs);
    w.group = (int)blockIdx.y / blocks;
    const int tile = ((int)blockIdx.y % blocks) * SCAN_WARPS + warp;
    w.r0 = w.seg * p.seg_rows;
    w.r1 = min(p.rows.rows, w.r0 + p.seg_rows);
    w.c0 = w.group * per + tile * K::CW;
    w.nch = min(K::CW, per - tile * K::CW);
    return w.nch > 0;
}

}  // namespace
}  // namespace selinv
