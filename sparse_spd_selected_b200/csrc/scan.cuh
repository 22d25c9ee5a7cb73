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

// Where a warp works: line and rows, channel group and channels.
struct ScanPlace {
    int64_t line;
    int r0, r1, seg, group, c0, nch;     // c0: first channel (of all d); nch <= CW of them
};

// Asynchronous copies of 4 and 8 bytes from global to shared memory.
SELINV_DEVINL void cp_async4(void *smem, const void *gmem)
{
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(s), "l"(gmem) : "memory");
}
SELINV_DEVINL void cp_async8(void *smem, const void *gmem)
{
    const unsigned s = static_cast<unsigned>(__cvta_generic_to_shared(smem));
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(s), "l"(gmem) : "memory");
}

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

// Starts copying CW channels (nch of them exist) of rows r .. r1 - 1, at most SCAN_R, into `to`.  FULL: all channels, all
// rows, on 16 bytes; straight code, since a few warps wait for nothing but their own instructions here.
template <int CW, bool FULL, class T>
SELINV_DEVINL void raw_fetch(T (*to)[CW], const T *from, const In &a, int r, int r1, int nch, int lane)
{
    const int stride = a.row;
    constexpr int E = 16 / (int)sizeof(T), LANES = CW / E, ROWS = 32 / LANES;
    static_assert(CW % E == 0 && LANES <= 32, "a warp copies whole rows");
    const int row = lane / LANES, e = (lane % LANES) * E;
    if (FULL) {
        const T *at = from + ((int64_t)(r + row) * stride + e);
        if (ROWS <= SCAN_R || row < SCAN_R) {
#pragma unroll
            for (int i = 0; i < SCAN_R; i += ROWS) cp_async16(&to[row + i][e], at + (int64_t)i * stride);
        }
        return;
    }
    const int nr = min(SCAN_R, r1 - r);
    if (a.wide && nch == CW) {
        const T *at = from + ((int64_t)(r + row) * stride + e);
#pragma unroll
        for (int i = 0; i < SCAN_R; i += ROWS)
            if (row + i < nr) cp_async16(&to[row + i][e], at + (int64_t)i * stride);
    } else if (a.words) {       // a word at a time, still asynchronously (4 x 1021 x 2051 x 16 in float: 178 us, 309 without)
        constexpr int W = sizeof(T) < 4 ? 2 : 1, ROW = CW / W;
#pragma unroll 2
        for (int i = lane; i < SCAN_R * ROW; i += 32) {
            const int t = i / ROW, c = (i % ROW) * W;
            if (t >= nr || c >= nch) continue;
            const T *at = from + ((int64_t)(r + t) * stride + c);
            if (c + W > nch)
                to[t][c] = *at;
            else if constexpr (sizeof(T) == 8)
                cp_async8(&to[t][c], at);
            else
                cp_async4(&to[t][c], at);
        }
    } else {                    // 16-bit elements on odd places
        for (int c = lane; c < nch; c += 32) {
#pragma unroll 4
            for (int i = 0; i < nr; ++i) to[i][c] = from[(int64_t)(r + i) * stride + c];
        }
    }
}
// The next such tile into L2.
template <class T>
SELINV_DEVINL void raw_prefetch(const T *from, int stride, int r, int r1, int nch, int lane)
{
    if (lane < SCAN_R && r + lane < r1 && nch > 0) prefetch_l2(from + (int64_t)(r + lane) * stride);
}
// The same of B or C [rows, n] into rows of NP, dealt out over THREADS threads; with zeros where states or rows are not
// there (they take part in sums over channels).  FULL: all rows, whole vectors; the states that are not there are zero
// already (raw_clear_n).
template <int THREADS, bool FULL, class T, int NP>
SELINV_DEVINL void raw_fetch_n(T (*to)[NP], const T *from, int stride, int r, int r1, int n, bool wide, int thread)
{
    constexpr int E = sizeof(T) == 2 ? 4 : 16 / (int)sizeof(T), ROW = NP / E;      // 8 or 16 bytes at a time
    const int nr = min(SCAN_R, r1 - r);
#pragma unroll
    for (int i = thread; i < SCAN_R * ROW; i += THREADS) {
        const int row = i / ROW, e = (i % ROW) * E;
        const T *at = from + ((int64_t)(r + row) * stride + e);
        if (FULL ? NP == n || e < n : (wide && row < nr && e + E <= n)) {
            if constexpr (sizeof(T) == 2)
                cp_async8(&to[row][e], at);
            else
                cp_async16(&to[row][e], at);
        } else if (!FULL) {
#pragma unroll
            for (int q = 0; q < E; ++q)
                to[row][e + q] = row < nr && e + q < n ? at[q] : Elem<T>::down((typename Elem<T>::C)0);
        }
    }
}
template <int THREADS, class T, int NP> SELINV_DEVINL void raw_clear_n(T (*to)[NP], int n, int thread)
{
    if (n == NP) return;
    for (int i = thread; i < SCAN_R * NP; i += THREADS) to[i / NP][i % NP] = Elem<T>::down((typename Elem<T>::C)0);
}
// Whether B's and C's states come in whole vectors.
template <class T> SELINV_DEVINL bool whole_n(int n) { return n % (sizeof(T) == 2 ? 4 : 16 / (int)sizeof(T)) == 0; }
// From there into the arithmetic type.
template <int THREADS, class T, int NP>
SELINV_DEVINL void raw_stage_n(typename Elem<T>::C (*to)[NP], const T (*from)[NP], int thread)
{
    constexpr int E = sizeof(T) == 2 ? 4 : 16 / (int)sizeof(T), ROW = NP / E;
#pragma unroll
    for (int i = thread; i < SCAN_R * ROW; i += THREADS) {
        const int row = i / ROW, e = (i % ROW) * E;
        Pack<T, E> v;
        v.load(&from[row][e], E, true);
        typename Elem<T>::C a[E];
#pragma unroll
        for (int q = 0; q < E; ++q) a[q] = v.get(q);
        put<E>(&to[row][e], a);
    }
}

// N states of a channel in a [d, n] array (p: the first of them, m of them exist, none where `in` is false): zero beyond;
// in pairs.
template <int N, class C> SELINV_DEVINL void load_states(const C *p, int m, bool in, typename Two<C>::V *v)
{
    if (in && m >= N && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        C t[N];
        get<N>(p, t);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) v[j] = make2(t[2 * j], t[2 * j + 1]);
        return;
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j)
        v[j] = make2(in && 2 * j < m ? p[2 * j] : (C)0, in && 2 * j + 1 < m ? p[2 * j + 1] : (C)0);
}
template <int N, class C> SELINV_DEVINL void store_states(C *p, int m, bool in, const typename Two<C>::V *v)
{
    if (!in) return;
    if (m >= N && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        C t[N];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) t[2 * j] = v[j].x, t[2 * j + 1] = v[j].y;
        put<N>(p, t);
        return;
    }
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        if (2 * j < m) p[2 * j] = v[j].x;
        if (2 * j + 1 < m) p[2 * j + 1] = v[j].y;
    }
}
// The J-th pair of a lane's states, of which m exist, with zeros for those that do not.  They have no inputs and are zero as
// it is, but for infinities: an infinite step or input times their B of zero is not a number.
template <class V> SELINV_DEVINL V real_states(V v, int J, int m)
{
    if (2 * J >= m) v.x = 0;
    if (2 * J + 1 >= m) v.y = 0;
    return v;
}
template <int N, class V> SELINV_DEVINL void zero_states(V *v)
{
#pragma unroll
    for (int j = 0; j < N / 2; ++j) v[j].x = v[j].y = 0;
}

// What the segments s, s + by, ... before `to` hand on to N states of one channel (own: their place in a [d, n] array):
// the first one's own, decayed by each later one's sum of steps and joined to that one's own.  The decays of a whole
// segment are taken in two halves of at most 2^127 (2^1023) each: steps that let a state grow (dt' A > 0) may leave
// that range although the state does not, and nothing times that is nothing.  Nor is a half below 2^-126 (2^-1022): what
// that leaves of a finite state is nothing to it, but zero times an infinite one is not a number.
template <int N, class C>
SELINV_DEVINL void scan_join(const ScanArgs &p, int64_t line, int s, int to, int by, int64_t channel, int64_t own, int m, bool in,
                             const typename Two<C>::V *A2, typename Two<C>::V *h)
{
    using V = typename Two<C>::V;
    const int64_t dn = p.d * p.n;
    const C *ends = static_cast<const C *>(p.ends) + line * p.segs * dn + own;
    const C *sums = static_cast<const C *>(p.sums) + line * p.segs * p.d + channel;
    load_states<N>(ends + s * dn, m, in, h);
    for (s += by; s != to; s += by) {
        V e[N / 2];
        load_states<N>(ends + s * dn, m, in, e);
        const C t = in ? sums[s * p.d] / 2 : (C)0, most = sizeof(C) == 4 ? 127 : 1023, least = 1 - most;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const V a = exp2_2(make2(fmax(fmin(t * A2[j].x, most), least), fmax(fmin(t * A2[j].y, most), least)));
            h[j] = fma2(a, mul2(a, h[j]), e[j]);
        }
    }
}

// Where this warp works, given a block's warps and a warp's channels; false: no channels are left for it.
SELINV_DEVINL bool scan_place(const ScanArgs &p, int warp, int warps, int cw, ScanPlace &w)
{
    const int per = (int)(p.d / p.groups), tiles = (per + cw - 1) / cw;
    const int blocks = (tiles + warps - 1) / warps;
    w.line = blockIdx.x / p.segs;
    w.seg = (int)(blockIdx.x % p.segs);
    w.group = (int)blockIdx.y / blocks;
    const int tile = ((int)blockIdx.y % blocks) * warps + warp;
    w.r0 = w.seg * p.seg_rows;
    w.r1 = piece_end(w.r0, p.seg_rows, p.rows.rows);
    w.c0 = w.group * per + tile * cw;
    w.nch = min(cw, per - tile * cw);
    return w.nch > 0;
}

}  // namespace
}  // namespace selinv
