// The short causal convolution of each channel along chains (sm_100a):
//   y_t = bias + sum_j weight_j x_{t-K+1+j}, then silu where asked,
// with the K - 1 rows before a sequence taken from its state or zero, and its
// last K - 1 inputs written as its new state.
//
// Bounded by memory: x is read and y written once.  A thread keeps E
// neighbouring channels (8 bytes of the 16-bit types, 16 of the others; pairs
// in one instruction) and runs down a chunk of rows with the last K - 1 inputs
// in registers, four rows at a time with the next four on their way, so that
// neighbouring threads read whole lines and each row is fetched once, but for
// the K - 1 rows before a chunk.  8 x 2048 x 4096, K = 4, bfloat16 with silu: 70
// us for 268 MB (0.58 of a plain copy's rate; the silu's power of two and
// reciprocal keep the special function unit half busy), the backward 137 us for
// 403 MB (0.45; it forms the output again).  Both run in a fraction of a wave more
// than they need: 1216 blocks where 740 are resident forward, 444 backward.  Single
// tokens: a channel, and so 2 bytes of the 16-bit types, per lane and load, the
// weights and the slots read by every row: 192 x 4096 takes 9 us, 2 of them memory.
#pragma once

#include "sequence.cuh"

namespace selinv {
namespace {

constexpr int CONV_THREADS = 128;
constexpr int CONV_U = 4;       // rows at a time

template <class T> struct ConvType {
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    static constexpr int E = sizeof(T) == 8 ? 2 : 4, EP = E / 2;
};

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
    w.r1 = piece_end(w.r0, p.chunk_rows, p.rows.rows);
    return true;
}

template <class T, int E> SELINV_DEVINL void unpack(const Pack<T, E> &q, typename ConvType<T>::V *v)
{
#pragma unroll
    for (int e = 0; e < E / 2; ++e) v[e] = make2(q.get(2 * e), q.get(2 * e + 1));
}
template <class T> SELINV_DEVINL void up_row(const T *p, int n, bool wide, typename ConvType<T>::V *v)
{
    Pack<T, ConvType<T>::E> q;
    q.load(p, n, wide);
    unpack(q, v);
}
template <class T> SELINV_DEVINL void down_row(T *p, int n, bool wide, const typename ConvType<T>::V *v)
{
    constexpr int E = ConvType<T>::E;
    typename Elem<T>::C t[E];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) t[2 * e] = v[e].x, t[2 * e + 1] = v[e].y;
    Pack<T, E> q;
    q.set(t);
    q.store(p, n, wide);
}

// CONV_U rows of E channels; one branch for all of them.
template <class T> SELINV_DEVINL void load_rows(const T *p, int stride, bool wide, Pack<T, ConvType<T>::E> *v)
{
    if (wide) {
#pragma unroll
        for (int i = 0; i < CONV_U; ++i) v[i].load(p + (int64_t)i * stride, ConvType<T>::E, true);
    } else {
#pragma unroll
        for (int i = 0; i < CONV_U; ++i) v[i].load(p + (int64_t)i * stride, ConvType<T>::E, false);
    }
}

// The K - 1 inputs before row r of the sequence that begins at row `start`.
template <class T, int K>
SELINV_DEVINL void conv_window(const ConvArgs &p, const T *x, int start, int64_t number, int r, int c, int n,
                               typename ConvType<T>::V (*win)[ConvType<T>::EP])
{
    const T *state = static_cast<const T *>(p.state);
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int at = r - (K - 1) + i;
        if (at >= start) {
            up_row(x + (int64_t)at * p.x.row, n, p.x.wide, win[i]);
        } else if (state) {
            up_row(state + (number * (K - 1) + (at - start + K - 1)) * p.d + c, n, false, win[i]);
        } else {
#pragma unroll
            for (int e = 0; e < ConvType<T>::EP; ++e) win[i][e].x = win[i][e].y = 0;
        }
    }
}

template <class T, int K>
SELINV_DEVINL void conv_weights(const ConvArgs &p, const ConvPlace &w, typename ConvType<T>::V (*wt)[ConvType<T>::EP],
                                typename ConvType<T>::V *bias)
{
    using C = typename Elem<T>::C;
    constexpr int E = ConvType<T>::E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const C v = e < w.n ? Elem<T>::up(static_cast<const T *>(p.weight)[(int64_t)(w.c + e) * K + j]) : (C)0;
            (e & 1 ? wt[j][e / 2].y : wt[j][e / 2].x) = v;
        }
        (e & 1 ? bias[e / 2].y : bias[e / 2].x) =
            e < w.n && p.bias ? Elem<T>::up(static_cast<const T *>(p.bias)[w.c + e]) : (C)0;
    }
}
// sum_j wt_j win_j + bias
template <int K, int EP, class V> SELINV_DEVINL void conv_taps(const V (*wt)[EP], const V *bias, const V (*win)[EP], V *v)
{
#pragma unroll
    for (int e = 0; e < EP; ++e) {
        v[e] = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) v[e] = fma2(wt[j][e], win[j][e], v[e]);
    }
}
template <int K, int M, int EP, class V> SELINV_DEVINL void conv_shift(V (*win)[EP])
{
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int e = 0; e < EP; ++e) win[j][e] = win[j + M][e];
}

template <class T, int K> __global__ void __launch_bounds__(CONV_THREADS) conv_kernel(const __grid_constant__ ConvArgs p)
{
    using C = typename Elem<T>::C;
    using V = typename ConvType<T>::V;
    constexpr int E = ConvType<T>::E, EP = ConvType<T>::EP, U = CONV_U;
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
    V wt[K][EP], bias[EP], win[K - 1 + U][EP];
    conv_weights<T, K>(p, w, wt, bias);
    int k = p.rows.find(w.r0), end = p.rows.end(k);
    conv_window<T, K>(p, x, p.rows.start(k), p.rows.number(k, w.line), w.r0, w.c, w.n, win);
    const bool whole = w.n == E;
    Pack<T, E> raw[U];
    bool ahead = false;         // raw holds the rows r on
    for (int r = w.r0; r < w.r1;) {
        const int last = min(w.r1, end);
        if (whole && r + U <= last) {
            if (!ahead) load_rows(x + (int64_t)r * p.x.row, p.x.row, p.x.wide, raw);
#pragma unroll
            for (int i = 0; i < U; ++i) unpack(raw[i], win[K - 1 + i]);
            ahead = r + 2 * U <= last;
            if (ahead) load_rows(x + (int64_t)(r + U) * p.x.row, p.x.row, p.x.wide, raw);
            V v[U][EP];
#pragma unroll
            for (int i = 0; i < U; ++i) conv_taps<K, EP>(wt, bias, win + i, v[i]);
            if (p.silu) {
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int e = 0; e < EP; ++e) v[i][e] = mul2(v[i][e], sigmoid2(v[i][e]));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) down_row(y + (int64_t)(r + i) * p.y.row, E, p.y.wide, v[i]);
            conv_shift<K, U, EP>(win);
            r += U;
        } else {
            V v[EP];
            up_row(x + (int64_t)r * p.x.row, w.n, p.x.wide, win[K - 1]);
            conv_taps<K, EP>(wt, bias, win, v);
            if (p.silu) {
#pragma unroll
                for (int e = 0; e < EP; ++e) v[e] = mul2(v[e], sigmoid2(v[e]));
            }
            down_row(y + (int64_t)r * p.y.row, w.n, p.y.wide, v);
            conv_shift<K, 1, EP>(win);
            ++r;
        }
        if (r == end) {
            if (state_out) {
                const int64_t at = p.rows.number(k, w.line) * (K - 1) * p.d + w.c;
#pragma unroll
                for (int i = 0; i < K - 1; ++i) down_row(state_out + at + i * p.d, w.n, false, win[i]);
            }
            if (r < w.r1) {
                ++k;
                end = p.rows.end(k);
                conv_window<T, K>(p, x, r, p.rows.number(k, w.line), r, w.c, w.n, win);
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
    using V = typename ConvType<T>::V;
    constexpr int E = ConvType<T>::E, EP = ConvType<T>::EP, U = CONV_U;
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
    // win: the inputs from K - 1 rows before row t on; ring: preb likewise
    V wt[K][EP], bias[EP], wsum[K][EP], bsum[EP], win[K - 1 + U][EP], ring[K - 1 + U][EP];
    const V none[EP] = {};
    conv_weights<T, K>(p, w, wt, bias);
#pragma unroll
    for (int e = 0; e < EP; ++e) {
        bsum[e] = none[e];
#pragma unroll
        for (int j = 0; j < K; ++j) wsum[j][e] = none[e];
    }
    const bool whole = w.n == E;
    if (w.r0 < w.r1) {
        int k = p.rows.find(w.r0);
        for (int r = w.r0; r < w.r1; ++k) {
            const int start = p.rows.start(k), end = p.rows.end(k);
            const int64_t number = p.rows.number(k, w.line);
            const bool head = start >= w.r0;                       // this chunk holds the sequence's first row
            const int m0 = head ? start - (K - 1) : w.r0, m1 = min(end, w.r1);
            conv_window<T, K>(p, x, start, number, r, w.c, w.n, win);
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int e = 0; e < EP; ++e) ring[j][e] = none[e];
            Pack<T, E> xr[U], yr[U];
            bool ahead = false;
            for (int t = r; t - (K - 1) < m1;) {
                // U rows from s on, none of them behind the sequence, no output of theirs a state's
                const auto plain = [&](int s) {
                    return whole && s + U <= end && (!stateb || s + U - K < end - (K - 1)) &&
                           (!stateb_out || s - (K - 1) >= start);
                };
                if (plain(t)) {
                    if (!ahead) {
                        load_rows(x + (int64_t)t * p.x.row, p.x.row, p.x.wide, xr);
                        load_rows(yb + (int64_t)t * p.yb.row, p.yb.row, p.yb.wide, yr);
                    }
                    V g[U][EP];
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        unpack(xr[i], win[K - 1 + i]);
                        unpack(yr[i], g[i]);
                    }
                    ahead = t + U - (K - 1) < m1 && plain(t + U);
                    if (ahead) {
                        load_rows(x + (int64_t)(t + U) * p.x.row, p.x.row, p.x.wide, xr);
                        load_rows(yb + (int64_t)(t + U) * p.yb.row, p.yb.row, p.yb.wide, yr);
                    }
                    if (p.silu) {
#pragma unroll
                        for (int i = 0; i < U; ++i) {
                            V v[EP];
                            conv_taps<K, EP>(wt, bias, win + i, v);
#pragma unroll
                            for (int e = 0; e < EP; ++e) g[i][e] = mul2(g[i][e], silu_slope2(v[e], sigmoid2(v[e])));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        const int m = t + i - (K - 1);
                        V v[EP];
#pragma unroll
                        for (int e = 0; e < EP; ++e) {
                            ring[K - 1 + i][e] = g[i][e];
                            v[e] = mul2(wt[K - 1][e], ring[i][e]);
#pragma unroll
                            for (int j = 1; j < K; ++j) v[e] = fma2(wt[K - 1 - j][e], ring[i + j][e], v[e]);
                        }
                        if (m >= max(m0, start) && m < m1) down_row(xb + (int64_t)m * p.xb.row, E, p.xb.wide, v);
                    }
                    const auto sum = [&](int i) {
#pragma unroll
                        for (int e = 0; e < EP; ++e) {
                            bsum[e] = add2(bsum[e], g[i][e]);
#pragma unroll
                            for (int j = 0; j < K; ++j) wsum[j][e] = fma2(g[i][e], win[i + j][e], wsum[j][e]);
                        }
                    };
                    if (t + U <= w.r1) {
#pragma unroll
                        for (int i = 0; i < U; ++i) sum(i);
                    } else {            // rows from r1 on are the next chunk's to sum
#pragma unroll
                        for (int i = 0; i < U; ++i)
                            if (t + i < w.r1) sum(i);
                    }
                    conv_shift<K, U, EP>(win);
                    conv_shift<K, U, EP>(ring);
                    t += U;
                    continue;
                }
                if (t < end) {
                    V g[EP];
                    up_row(x + (int64_t)t * p.x.row, w.n, p.x.wide, win[K - 1]);
                    up_row(yb + (int64_t)t * p.yb.row, w.n, p.yb.wide, g);
                    if (p.silu) {
                        V v[EP];
                        conv_taps<K, EP>(wt, bias, win, v);
#pragma unroll
                        for (int e = 0; e < EP; ++e) g[e] = mul2(g[e], silu_slope2(v[e], sigmoid2(v[e])));
                    }
#pragma unroll
                    for (int e = 0; e < EP; ++e) {
                        ring[K - 1][e] = g[e];
                        if (t < w.r1) {
                            bsum[e] = add2(bsum[e], g[e]);
#pragma unroll
                            for (int j = 0; j < K; ++j) wsum[j][e] = fma2(g[e], win[j][e], wsum[j][e]);
                        }
                    }
                    conv_shift<K, 1, EP>(win);
                } else {
#pragma unroll
                    for (int e = 0; e < EP; ++e) ring[K - 1][e] = none[e];
                }
                const int m = t - (K - 1);
                if (m >= m0) {
                    V v[EP];
#pragma unroll
                    for (int e = 0; e < EP; ++e) {
                        v[e] = mul2(wt[K - 1][e], ring[0][e]);
#pragma unroll
                        for (int j = 1; j < K; ++j) v[e] = fma2(wt[K - 1 - j][e], ring[j][e], v[e]);
                    }
                    const int j = m - (end - (K - 1));             // the row of the final state that is this input
                    if (stateb && j >= 0) {
                        V s[EP];
                        up_row(stateb + (number * (K - 1) + j) * p.d + w.c, w.n, false, s);
#pragma unroll
                        for (int e = 0; e < EP; ++e) v[e] = add2(v[e], s[e]);
                    }
                    if (m >= start)
                        down_row(xb + (int64_t)m * p.xb.row, w.n, p.xb.wide, v);
                    else if (stateb_out)
                        down_row(stateb_out + (number * (K - 1) + (m - start + K - 1)) * p.d + w.c, w.n, false, v);
                }
                conv_shift<K, 1, EP>(ring);
                ++t;
            }
            r = m1;
        }
    }
    C *part = static_cast<C *>(p.part) + (w.line * p.chunks + w.chunk) * (K + 1) * p.d + w.c;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (e < w.n) {
#pragma unroll
            for (int j = 0; j < K; ++j) part[j * p.d + e] = e & 1 ? wsum[j][e / 2].y : wsum[j][e / 2].x;
            part[K * p.d + e] = e & 1 ? bsum[e / 2].y : bsum[e / 2].x;
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
#pragma unroll 8
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

// The slot of a step's row r, or -1 where there is none: a slot of -1 skips the row, one outside the cache is reported.
SELINV_DEVINL int64_t step_slot(const int32_t *index, int64_t r, int64_t slots)
{
    if (!index) return r;
    const int32_t slot = index[r];
    return slot >= 0 && slot < slots ? slot : -1;
}
// Whether the row may write to it: no earlier row names the same slot.  Reports the row's status.  Every thread of the
// block calls it, once its loads are on their way.
SELINV_DEVINL bool step_first(const int32_t *index, int32_t *info, int64_t r, int64_t slot, bool reports)
{
    if (!index) return true;
    bool twice = false;
    if (slot >= 0)
        for (int i = threadIdx.x; i < (int)r; i += blockDim.x) twice |= index[i] == (int)slot;
    twice = __syncthreads_or(twice);
    if (reports && info && threadIdx.x == 0)
        info[r] = twice ? STEP_TWICE : slot < 0 && index[r] != -1 ? STEP_RANGE : STEP_OK;
    return slot >= 0 && !twice;
}

// One row per sequence over a cache of states [slots, K - 1, d].
template <class T, int K>
__global__ void __launch_bounds__(CONV_THREADS) conv_step_kernel(const __grid_constant__ ConvStepArgs p)
{
    using C = typename Elem<T>::C;
    const unsigned blocks = (unsigned)((p.d + CONV_THREADS - 1) / CONV_THREADS), row = blockIdx.x / blocks;
    const int64_t r = row;
    const int c = (int)(blockIdx.x - row * blocks) * CONV_THREADS + threadIdx.x;
    const int64_t slot = step_slot(p.index, r, p.slots);
    const bool in = c < p.d;
    T win[K];
    C wt[K], bias = 0;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        win[j] = Elem<T>::down((C)0);
        wt[j] = 0;
    }
    if (in && slot >= 0) {
        const T *at = static_cast<const T *>(p.cache) + slot * (K - 1) * p.d + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) win[j] = at[j * p.d];
        win[K - 1] = static_cast<const T *>(p.x)[r * p.x_row + c];
        if (p.bias) bias = Elem<T>::up(static_cast<const T *>(p.bias)[c]);
#pragma unroll
        for (int j = 0; j < K; ++j) wt[j] = Elem<T>::up(static_cast<const T *>(p.weight)[c * K + j]);
    }
    const bool ours = step_first(p.index, p.info, r, slot, blockIdx.x == row * blocks);
    if (!in) return;
    C v = bias;
#pragma unroll
    for (int j = 0; j < K; ++j) v += wt[j] * Elem<T>::up(win[j]);
    if (p.silu) v *= sigmoid_(v);
    static_cast<T *>(p.y)[r * p.y_row + c] = Elem<T>::down(ours ? v : (C)0);
    if (ours) {
        T *out = static_cast<T *>(p.cache_out) + slot * (K - 1) * p.d + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) out[j * p.d] = win[j + 1];
    }
}

template <class T, int K> cudaError_t conv_run(const ConvArgs &p, cudaStream_t s)
{
    constexpr int E = ConvType<T>::E;
    const int64_t threads = (p.d + E - 1) / E * p.lines * p.chunks;
    conv_kernel<T, K><<<(unsigned)((threads + CONV_THREADS - 1) / CONV_THREADS), CONV_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}
template <class T, int K> cudaError_t conv_backward_run(const ConvArgs &p, cudaStream_t s)
{
    constexpr int E = ConvType<T>::E;
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
