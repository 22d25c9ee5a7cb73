// The short causal convolution of each channel along chains (sm_100a):
//   y_t = bias + sum_j weight_j x_{t-K+1+j}, then silu where asked,
// with the K - 1 rows before a sequence taken from its state or zero, and its
// last K - 1 inputs written as its new state.
//
// Bounded by memory: x is read and y written once.  A thread keeps 16 bytes
// of channels (E of them) and runs down a chunk of rows with the last K - 1
// inputs in registers, so that neighbouring threads read whole lines and each
// row is fetched once, but for the K - 1 rows before a chunk.
#pragma once

#include "sequence.cuh"

namespace selinv {
namespace {

constexpr int CONV_THREADS = 128;

// A thread's chunk: line, rows [r0, r1), channels [c, c + n).
struct ConvPlace {
    int64_t line;
    int r0, r1, chunk, c, n;
};
template <int E> SELINV_DEVINL bool conv_place(const ConvArgs &p, ConvPlace &w)
{
    const int64_t vecs = (p.d + E - 1) / E, id = (int64_t)blockIdx.x * CONV_THREADS + threadIdx.x;
    const int64_t rest = id / vecs;
    if (rest >= p.lines * p.chunks) return false;
    w.c = (int)(id % vecs) * E;
    w.n = (int)min((int64_t)E, p.d - w.c);
    w.line = rest / p.chunks;
    w.chunk = (int)(rest % p.chunks);
    w.r0 = w.chunk * p.chunk_rows;
    w.r1 = min(p.rows.rows, w.r0 + p.chunk_rows);
    return true;
}

template <class T, int E> SELINV_DEVINL void up_row(const T *p, int n, bool wide, typename Elem<T>::C *v)
{
    Pack<T, E> q;
    q.load(p, n, wide);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = q.get(e);
}
template <class T, int E> SELINV_DEVINL void down_row(T *p, int n, bool wide, const typename Elem<T>::C *v)
{
    Pack<T, E> q;
    q.set(v);
    q.store(p, n, wide);
}

// The K - 1 inputs before row r of the sequence that begins at row `start`.
template <class T, int K, int E>
SELINV_DEVINL void conv_window(const ConvArgs &p, const T *x, int start, int64_t number, int r, int c, int n,
                               typename Elem<T>::C (*win)[E])
{
    const T *state = static_cast<const T *>(p.state);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int at = r - (K - 1) + i;
        if (at >= start) {
            up_row<T, E>(x + (int64_t)at * p.x.row, n, p.x.wide, win[i]);
        } else if (state) {
            up_row<T, E>(state + (number * (K - 1) + (at - start + K - 1)) * p.d + c, n, false, win[i]);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) win[i][e] = 0;
        }
    }
}

template <class T, int K, int E>
SELINV_DEVINL void conv_weights(const ConvArgs &p, const ConvPlace &w, typename Elem<T>::C (*wt)[E],
                                typename Elem<T>::C *bias)
{
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            wt[j][e] = e < w.n ? Elem<T>::up(static_cast<const T *>(p.weight)[(int64_t)(w.c + e) * K + j]) : 0;
        bias[e] = e < w.n && p.bias ? Elem<T>::up(static_cast<const T *>(p.bias)[w.c + e]) : 0;
    }
}

template <class T, int K> __global__ void __launch_bounds__(CONV_THREADS) conv_kernel(const __grid_constant__ ConvArgs p)
{
    using C = typename Elem<T>::C;
    constexpr int E = 16 / (int)sizeof(T), U = 4;
    ConvPlace w;
    if (!conv_place<E>(p, w)) return;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c;
    T *y = static_cast<T *>(p.y.p) + w.line * p.y.line + w.c;
    T *state_out = static_cast<T *>(p.state_out);
    if (state_out && p.rows.table && w.chunk == 0) {    // sequences without rows end as they began
        const T *state = static_cast<const T *>(p.state);
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.empty(e) * (K - 1) * p.d + w.c;
            for (int i = 0; i < K - 1; ++i)
                for (int q = 0; q < w.n; ++q)
                    state_out[at + i * p.d + q] = state ? state[at + i * p.d + q] : Elem<T>::down((C)0);
        }
    }
    if (w.r0 >= w.r1) return;
    C wt[K][E], bias[E], win[K - 1 + U][E];
    conv_weights<T, K, E>(p, w, wt, bias);
    int k = p.rows.find(w.r0), end = p.rows.end(k);
    conv_window<T, K, E>(p, x, p.rows.start(k), p.rows.number(k, w.line), w.r0, w.c, w.n, win);
    for (int r = w.r0; r < w.r1;) {
        const int m = min(U, min(w.r1, end) - r);
        if (m == U) {
            Pack<T, E> raw[U];
#pragma unroll
            for (int i = 0; i < U; ++i) raw[i].load(x + (int64_t)(r + i) * p.x.row, w.n, p.x.wide);
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) win[K - 1 + i][e] = raw[i].get(e);
#pragma unroll
            for (int i = 0; i < U; ++i) {
                C v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] = bias[e];
#pragma unroll
                    for (int j = 0; j < K; ++j) v[e] += wt[j][e] * win[i + j][e];
                    if (p.silu) v[e] *= sigmoid_(v[e]);
                }
                down_row<T, E>(y + (int64_t)(r + i) * p.y.row, w.n, p.y.wide, v);
            }
#pragma unroll
            for (int i = 0; i < K - 1; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) win[i][e] = win[U + i][e];
        } else {
            for (int i = 0; i < m; ++i) {
                C v[E];
                up_row<T, E>(x + (int64_t)(r + i) * p.x.row, w.n, p.x.wide, win[K - 1]);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] = bias[e];
#pragma unroll
                    for (int j = 0; j < K; ++j) v[e] += wt[j][e] * win[j][e];
                    if (p.silu) v[e] *= sigmoid_(v[e]);
                }
                down_row<T, E>(y + (int64_t)(r + i) * p.y.row, w.n, p.y.wide, v);
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e) win[j][e] = win[j + 1][e];
            }
        }
        r += m;
        if (r == end) {
            if (state_out) {
                const int64_t at = p.rows.number(k, w.line) * (K - 1) * p.d + w.c;
#pragma unroll
                for (int i = 0; i < K - 1; ++i) down_row<T, E>(state_out + at + i * p.d, w.n, false, win[i]);
            }
            if (r < w.r1) {
                ++k;
                end = p.rows.end(k);
                conv_window<T, K, E>(p, x, r, p.rows.number(k, w.line), r, w.c, w.n, win);
            }
        }
    }
}

// Backward: preb_t = yb_t silu'(pre_t) with pre_t formed again, xb_m = sum_j weight_j preb_{m+K-1-j} over the rows of
// m's own sequence, weightb_j = sum_t preb_t x_{t-K+1+j}.  Runs down the chunk like the forward, K - 1 rows further,
// and writes the row K - 1 behind; the parameters' sums go out per chunk, in a fixed order.
template <class T, int K>
__global__ void __launch_bounds__(CONV_THREADS) conv_backward_kernel(const __grid_constant__ ConvArgs p)
{
    using C = typename Elem<T>::C;
    constexpr int E = 16 / (int)sizeof(T);
    ConvPlace w;
    if (!conv_place<E>(p, w)) return;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c;
    const T *yb = static_cast<const T *>(p.yb.p) + w.line * p.yb.line + w.c;
    T *xb = static_cast<T *>(p.xb.p) + w.line * p.xb.line + w.c;
    const T *stateb = static_cast<const T *>(p.stateb);
    T *stateb_out = static_cast<T *>(p.stateb_out);
    if (stateb_out && p.rows.table && w.chunk == 0) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.empty(e) * (K - 1) * p.d + w.c;
            for (int i = 0; i < K - 1; ++i)
                for (int q = 0; q < w.n; ++q)
                    stateb_out[at + i * p.d + q] = stateb ? stateb[at + i * p.d + q] : Elem<T>::down((C)0);
        }
    }
    C wt[K][E], bias[E], wsum[K][E], bsum[E], win[K][E], ring[K][E];
    conv_weights<T, K, E>(p, w, wt, bias);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        bsum[e] = 0;
#pragma unroll
        for (int j = 0; j < K; ++j) wsum[j][e] = 0;
    }
    if (w.r0 < w.r1) {
        int k = p.rows.find(w.r0);
        for (int r = w.r0; r < w.r1; ++k) {
            const int start = p.rows.start(k), end = p.rows.end(k);
            const int64_t number = p.rows.number(k, w.line);
            const bool head = start >= w.r0;                       // this chunk holds the sequence's first row
            const int m0 = head ? start - (K - 1) : w.r0, m1 = min(end, w.r1);
            conv_window<T, K, E>(p, x, start, number, r, w.c, w.n, win);
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) ring[j][e] = 0;
            for (int t = r; t - (K - 1) < m1; ++t) {
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int e = 0; e < E; ++e) ring[j][e] = ring[j + 1][e];
                if (t < end) {
                    C g[E];
                    up_row<T, E>(x + (int64_t)t * p.x.row, w.n, p.x.wide, win[K - 1]);
                    up_row<T, E>(yb + (int64_t)t * p.yb.row, w.n, p.yb.wide, g);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (p.silu) {
                            C v = bias[e];
#pragma unroll
                            for (int j = 0; j < K; ++j) v += wt[j][e] * win[j][e];
                            g[e] *= silu_slope(v, sigmoid_(v));
                        }
                        ring[K - 1][e] = g[e];
                        if (t < w.r1) {
                            bsum[e] += g[e];
#pragma unroll
                            for (int j = 0; j < K; ++j) wsum[j][e] += g[e] * win[j][e];
                        }
                    }
#pragma unroll
                    for (int j = 0; j < K - 1; ++j)
#pragma unroll
                        for (int e = 0; e < E; ++e) win[j][e] = win[j + 1][e];
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) ring[K - 1][e] = 0;
                }
                const int m = t - (K - 1);
                if (m < m0) continue;
                C v[E];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] = 0;
#pragma unroll
                    for (int j = 0; j < K; ++j) v[e] += wt[j][e] * ring[K - 1 - j][e];
                }
                const int j = m - (end - (K - 1));             // the row of the final state that is this input
                if (stateb && j >= 0) {
                    C s[E];
                    up_row<T, E>(stateb + (number * (K - 1) + j) * p.d + w.c, w.n, false, s);
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] += s[e];
                }
                if (m >= start)
                    down_row<T, E>(xb + (int64_t)m * p.xb.row, w.n, p.xb.wide, v);
                else if (stateb_out)
                    down_row<T, E>(stateb_out + (number * (K - 1) + (m - start + K - 1)) * p.d + w.c, w.n, false, v);
            }
            r = m1;
        }
    }
    C *part = static_cast<C *>(p.part) + (w.line * p.chunks + w.chunk) * (K + 1) * p.d + w.c;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < w.n) {
#pragma unroll
            for (int j = 0; j < K; ++j) part[j * p.d + e] = wsum[j][e];
            part[K * p.d + e] = bsum[e];
        }
}

// weightb [d, k] and biasb [d] from the chunks' sums: 32 channels of one tap per block, 8 strands of chunks, each
// strand and then the strands in order.
template <class C> __global__ void __launch_bounds__(256) conv_params_kernel(const __grid_constant__ ConvArgs p)
{
    __shared__ C s[8][32];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x % 32, count = p.lines * p.chunks;
    const int j = blockIdx.y, strand = threadIdx.x / 32;
    C v = 0;
    if (c < p.d)
        for (int64_t i = strand; i < count; i += 8)
            v += static_cast<const C *>(p.part)[(i * (p.k + 1) + j) * p.d + c];
    s[strand][threadIdx.x % 32] = v;
    __syncthreads();
    if (strand == 0 && c < p.d) {
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
        if (j < p.k)
            static_cast<C *>(p.weightb)[c * p.k + j] = v;
        else if (p.biasb)
            static_cast<C *>(p.biasb)[c] = v;
    }
}

// What a step does with row r: its slot, or -1 where it leaves the cache alone.  A slot of -1 skips the row; one
// outside the cache, or one that an earlier row names too, is reported.  Every thread of the block calls it.
SELINV_DEVINL int64_t step_slot(const int32_t *index, int32_t *info, int64_t r, int64_t slots, bool reports)
{
    if (!index) return r;
    const int32_t slot = index[r];
    int32_t status = STEP_OK;
    bool twice = false;
    if (slot < -1 || slot >= slots) status = STEP_RANGE;
    if (slot >= 0)
        for (int64_t i = threadIdx.x; i < r; i += blockDim.x) twice |= index[i] == slot;
    if (__syncthreads_or(twice)) status = STEP_TWICE;
    if (reports && info && threadIdx.x == 0) info[r] = status;
    return status == STEP_OK ? slot : -1;
}

// One row per sequence over a cache of states [slots, K - 1, d].
template <class T, int K>
__global__ void __launch_bounds__(CONV_THREADS) conv_step_kernel(const __grid_constant__ ConvStepArgs p)
{
    using C = typename Elem<T>::C;
    const int64_t blocks = (p.d + CONV_THREADS - 1) / CONV_THREADS, r = blockIdx.x / blocks;
    const int64_t c = (blockIdx.x % blocks) * CONV_THREADS + threadIdx.x;
    const int64_t slot = step_slot(p.index, p.info, r, p.slots, blockIdx.x % blocks == 0);
    if (c >= p.d) return;
    T *y = static_cast<T *>(p.y) + r * p.y_row + c;
    if (slot < 0) {
        *y = Elem<T>::down((C)0);
        return;
    }
    const T *in = static_cast<const T *>(p.cache) + slot * (K - 1) * p.d + c;
    T *out = static_cast<T *>(p.cache_out) + slot * (K - 1) * p.d + c;
    T win[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j] = in[j * p.d];
    win[K - 1] = static_cast<const T *>(p.x)[r * p.x_row + c];
    C v = p.bias ? Elem<T>::up(static_cast<const T *>(p.bias)[c]) : (C)0;
#pragma unroll
    for (int j = 0; j < K; ++j) v += Elem<T>::up(static_cast<const T *>(p.weight)[c * K + j]) * Elem<T>::up(win[j]);
    if (p.silu) v *= sigmoid_(v);
    *y = Elem<T>::down(v);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) out[j * p.d] = win[j + 1];
}

template <class T, int K> cudaError_t conv_run(const ConvArgs &p, cudaStream_t s)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t threads = (p.d + E - 1) / E * p.lines * p.chunks;
    conv_kernel<T, K><<<(unsigned)((threads + CONV_THREADS - 1) / CONV_THREADS), CONV_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}
template <class T, int K> cudaError_t conv_backward_run(const ConvArgs &p, cudaStream_t s)
{
    constexpr int E = 16 / (int)sizeof(T);
    const int64_t threads = (p.d + E - 1) / E * p.lines * p.chunks;
    conv_backward_kernel<T, K><<<(unsigned)((threads + CONV_THREADS - 1) / CONV_THREADS), CONV_THREADS, 0, s>>>(p);
    const dim3 grid((unsigned)((p.d + 31) / 32), (unsigned)(K + 1));
    conv_params_kernel<typename Elem<T>::C><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <class T, int K> cudaError_t conv_step_run(const ConvStepArgs &p, cudaStream_t s)
{
    const int64_t blocks = (p.d + CONV_THREADS - 1) / CONV_THREADS * p.batch;
    conv_step_kernel<T, K><<<(unsigned)blocks, CONV_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
