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

// A warp's tile: TD channels x TN states in each thread, LN groups of LD lanes along the states: lane = nl * LD + dl
// holds the channels dl * TD on and the states nl * TN on, so that the lanes that read or write shared memory together
// lie side by side along the channels.  The same lane converts rows nl, nl + LN, ... of its channels.
template <class T_, int TD_, int TN_, int NP_> struct ScanTile {
    using T = T_;
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    static constexpr int TD = TD_, TN = TN_, NP = NP_, LN = NP / TN, LD = 32 / LN, CW = LD * TD, TP = TD / 2;
    static constexpr int PER = (SCAN_R + LN - 1) / LN;           // rows that a lane converts
    // elements of B and C a lane converts at a time
    static constexpr int EB = sizeof(T) == 8 ? 2 : 4, BVECS = SCAN_R * NP / EB, BPER = (BVECS + 31) / 32;
    static_assert(LN * LD == 32 && TD * sizeof(C) == 16, "a lane's channels are 16 bytes of shared memory");
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

template <int N> SELINV_DEVINL void put(float *p, const float2 *v)
{
    float t[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) t[2 * i] = v[i].x, t[2 * i + 1] = v[i].y;
    put<2 * N>(p, t);
}
template <int N> SELINV_DEVINL void put(double *p, const double2 *v)
{
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<double2 *>(p + 2 * i) = v[i];
}

// A lane's rows of a tile of an array [rows, channels] (p: the lane's first channel; n of them exist).
template <class K> struct ScanLoad {
    using T = typename K::T;
    Pack<T, K::TD> v[K::PER];
    SELINV_DEVINL void load(const T *p, int64_t stride, int64_t r0, int64_t r1, int n, bool wide, int nl)
    {
#pragma unroll
        for (int i = 0; i < K::PER; ++i) {
            const int row = nl + K::LN * i;
            v[i].clear();
            if (row < SCAN_R && r0 + row < r1) v[i].load(p + (r0 + row) * stride, n, wide);
        }
    }
};
// The same of B or C [rows, n]: vectors of EB states, dealt out over `LANES` lanes.
template <class K, int LANES> struct ScanLoadN {
    using T = typename K::T;
    static constexpr int PER = (K::BVECS + LANES - 1) / LANES;
    Pack<T, K::EB> v[PER];
    SELINV_DEVINL static int row(int lane, int i) { return (lane + LANES * i) / (K::NP / K::EB); }
    SELINV_DEVINL static int first(int lane, int i) { return (lane + LANES * i) % (K::NP / K::EB) * K::EB; }
    SELINV_DEVINL void load(const T *p, int64_t stride, int64_t r0, int64_t r1, int n, bool wide, int lane)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = row(lane, i), e = first(lane, i);
            v[i].clear();
            if (r < SCAN_R && r0 + r < r1) v[i].load(p + (r0 + r) * stride + e, n - e, wide);
        }
    }
    // into shared memory, each value twice: a pair of equal ones for two channels
    template <class C> SELINV_DEVINL void stage(C (*to)[2 * K::NP], int lane) const
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = row(lane, i);
            if (r >= SCAN_R) break;
            C a[2 * K::EB];
#pragma unroll
            for (int e = 0; e < K::EB; ++e) a[2 * e] = a[2 * e + 1] = v[i].get(e);
            put<2 * K::EB>(&to[r][2 * first(lane, i)], a);
        }
    }
};

// The thread's TD x TN part of a [d, n] array (p: the warp's first channel); what lies outside is zero.
template <class K> SELINV_DEVINL bool part_wide(const void *p, int n, int nch)
{
    return n == K::NP && nch == K::CW && reinterpret_cast<uintptr_t>(p) % (K::TN * sizeof(typename K::C)) == 0;
}
template <class K> SELINV_DEVINL void load_part(const typename K::C *p, int n, int nch, int lane, typename K::V (*v)[K::TN])
{
    using C = typename K::C;
    const int d0 = (lane % K::LD) * K::TD, n0 = (lane / K::LD) * K::TN;
    if (K::TN * sizeof(C) >= 8 && part_wide<K>(p, n, nch)) {
#pragma unroll
        for (int d = 0; d < K::TD; ++d) {
            C t[K::TN + 1];
            if constexpr (K::TN >= 2) get<K::TN>(p + (int64_t)(d0 + d) * n + n0, t);
#pragma unroll
            for (int j = 0; j < K::TN; ++j) (d & 1 ? v[d / 2][j].y : v[d / 2][j].x) = t[j];
        }
        return;
    }
#pragma unroll
    for (int d = 0; d < K::TD; ++d)
#pragma unroll
        for (int j = 0; j < K::TN; ++j)
            (d & 1 ? v[d / 2][j].y : v[d / 2][j].x) =
                n0 + j < n && d0 + d < nch ? p[(int64_t)(d0 + d) * n + n0 + j] : (C)0;
}
template <class K> SELINV_DEVINL void store_part(typename K::C *p, int n, int nch, int lane, typename K::V (*v)[K::TN])
{
    using C = typename K::C;
    const int d0 = (lane % K::LD) * K::TD, n0 = (lane / K::LD) * K::TN;
    if (K::TN * sizeof(C) >= 8 && part_wide<K>(p, n, nch)) {
#pragma unroll
        for (int d = 0; d < K::TD; ++d) {
            C t[K::TN + 1];
#pragma unroll
            for (int j = 0; j < K::TN; ++j) t[j] = d & 1 ? v[d / 2][j].y : v[d / 2][j].x;
            if constexpr (K::TN >= 2) put<K::TN>(p + (int64_t)(d0 + d) * n + n0, t);
        }
        return;
    }
#pragma unroll
    for (int d = 0; d < K::TD; ++d)
#pragma unroll
        for (int j = 0; j < K::TN; ++j)
            if (n0 + j < n && d0 + d < nch)
                p[(int64_t)(d0 + d) * n + n0 + j] = d & 1 ? v[d / 2][j].y : v[d / 2][j].x;
}
template <class K> SELINV_DEVINL void zero_part(typename K::V (*v)[K::TN])
{
#pragma unroll
    for (int q = 0; q < K::TP; ++q)
#pragma unroll
        for (int j = 0; j < K::TN; ++j) v[q][j] = make2((typename K::C)0, (typename K::C)0);
}
// A log2 e, and whether every entry of the warp is a plain decay (finite, at most zero).
template <class K>
SELINV_DEVINL bool load_decay(const void *A, int64_t part, int n, int nch, int lane, typename K::V (*v)[K::TN])
{
    using C = typename K::C;
    load_part<K>(static_cast<const C *>(A) + part, n, nch, lane, v);
    bool plain = true;
#pragma unroll
    for (int q = 0; q < K::TP; ++q)
#pragma unroll
        for (int j = 0; j < K::TN; ++j) {
            v[q][j] = mul2(v[q][j], make2(log2e<C>(), log2e<C>()));
            plain = plain && v[q][j].x <= 0 && v[q][j].y <= 0 && v[q][j].x > -(C)1e30 && v[q][j].y > -(C)1e30;
        }
    return __all_sync(FULL_MASK, plain);
}

// Which pairs of a thread's tile take their powers of two from the FMA pipe: SCAN_POLY of 8, evenly spread over the
// pairs of four rows.
constexpr int SCAN_POLY = 3;
template <class K> __host__ __device__ constexpr bool poly_pair(int row, int q, int j)
{
    return ((row * K::TP * K::TN + q * K::TN + j) * SCAN_POLY) % 8 + SCAN_POLY >= 8;
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

// Channels c + 2 q and the next of an array [d] or null (zero); nd of the lane's channels exist.
template <class K> SELINV_DEVINL typename K::V pair_of(const void *a, int64_t c, int nd, int q)
{
    using C = typename K::C;
    const C *p = static_cast<const C *>(a) + c + 2 * q;
    return make2(a && 2 * q < nd ? p[0] : (C)0, a && 2 * q + 1 < nd ? p[1] : (C)0);
}

// f(kind, q, j) for every pair of a thread's tile, `kind` telling at compile time where its power of two comes from.
template <class K, bool POLY, int ROW, int I = 0, class F> SELINV_DEVINL void scan_pairs(F f)
{
    if constexpr (I < K::TP * K::TN) {
        constexpr int q = I % K::TP, j = I / K::TP;
        f(std::integral_constant<bool, POLY && poly_pair<K>(ROW, q, j)>(), q, j);
        scan_pairs<K, POLY, ROW, I + 1>(f);
    }
}

// What the segments s, s + by, ... before `to` hand on: the first one's own, decayed by each later one's sum of steps and
// joined to that one's own.
template <class K>
SELINV_DEVINL void scan_join(const ScanArgs &p, const ScanPlace &w, int s, int to, int by, int lane,
                             const typename K::V (*A2)[K::TN], typename K::V (*h)[K::TN])
{
    using C = typename K::C;
    using V = typename K::V;
    const int64_t dn = p.d * p.n, part = (int64_t)w.c0 * p.n;
    const int d0 = (lane % K::LD) * K::TD;
    const C *ends = static_cast<const C *>(p.ends) + w.line * p.segs * dn + part;
    const C *sums = static_cast<const C *>(p.sums) + w.line * p.segs * p.d;
    load_part<K>(ends + s * dn, p.n, w.nch, lane, h);
    for (s += by; s != to; s += by) {
        V e[K::TP][K::TN];
        load_part<K>(ends + s * dn, p.n, w.nch, lane, e);
#pragma unroll
        for (int q = 0; q < K::TP; ++q) {
            const V t = pair_of<K>(sums + s * p.d, w.c0 + d0, w.nch - d0, q);
#pragma unroll
            for (int j = 0; j < K::TN; ++j) h[q][j] = fma2(decay2<false>(mul2(t, A2[q][j])), h[q][j], e[q][j]);
        }
    }
}
template <class K>
SELINV_DEVINL void scan_leave(const ScanArgs &p, const ScanPlace &w, int lane, typename K::V (*h)[K::TN], const typename K::V *total)
{
    using C = typename K::C;
    const int64_t at = w.line * p.segs + w.seg;
    const int d0 = (lane % K::LD) * K::TD;
    store_part<K>(static_cast<C *>(p.ends) + (at * p.d + w.c0) * p.n, p.n, w.nch, lane, h);
    if (lane / K::LD == 0) {
        C *sums = static_cast<C *>(p.sums) + at * p.d + w.c0;
#pragma unroll
        for (int q = 0; q < K::TP; ++q) {
            if (d0 + 2 * q < w.nch) sums[d0 + 2 * q] = total[q].x;
            if (d0 + 2 * q + 1 < w.nch) sums[d0 + 2 * q + 1] = total[q].y;
        }
    }
}

}  // namespace
}  // namespace selinv
