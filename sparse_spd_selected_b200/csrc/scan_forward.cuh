// Forward of the selective scan.  One warp works on CW channels of one
// segment of a line, row after row: a thread keeps TD x TN states in
// registers, packed in pairs of channels, and leaves the TD partial sums of y
// in shared memory, where the lanes that finish the rows (D x, the gate, the
// rounding) add the LN parts.  Rows are staged SCAN_R at a time in the warp's
// own shared memory (steps, steps times x, B and C as pairs of equal values);
// the next rows' loads are in flight meanwhile.  No two warps wait for one
// another.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

template <class K> struct ScanFwdSmem {
    using C = typename K::C;
    C dt[SCAN_R][K::CW], u[SCAN_R][K::CW], y[SCAN_R][K::LN][K::CW];
    C b[SCAN_R][2 * K::NP], c[SCAN_R][2 * K::NP];
};
template <class K> constexpr bool scan_fwd_aligned =
    sizeof(ScanFwdSmem<K>) % 16 == 0 && offsetof(ScanFwdSmem<K>, b) % 16 == 0 && offsetof(ScanFwdSmem<K>, y) % 16 == 0 &&
    offsetof(ScanFwdSmem<K>, u) % 16 == 0 && offsetof(ScanFwdSmem<K>, c) % 16 == 0;

// Row t of the tile: states on, and (MAIN) this thread's parts of y.  ROW: t's place among four.
template <class K, bool MAIN, bool POLY, int ROW>
SELINV_DEVINL void scan_row(ScanFwdSmem<K> &sm, int t, int d0, int n0, int nl, int n, const typename K::V (*A2)[K::TN],
                            typename K::V (*h)[K::TN], typename K::V *total)
{
    using C = typename K::C;
    using V = typename K::V;
    V dt2[K::TP], u2[K::TP], b2[K::TN], c2[K::TN], y2[K::TP];
    get<K::TP>(&sm.dt[t][d0], dt2);
    get<K::TP>(&sm.u[t][d0], u2);
    get<K::TN>(&sm.b[t][2 * n0], b2);
    if (MAIN) get<K::TN>(&sm.c[t][2 * n0], c2);
    scan_pairs<K, POLY, ROW>([&](auto poly, int q, int j) {
        const V a = decay2<poly.value>(mul2(dt2[q], A2[q][j]));
        h[q][j] = fma2(a, h[q][j], mul2(u2[q], b2[j]));
    });
    if (n < K::NP) {        // an infinite x must not reach y through a state that is not there
#pragma unroll
        for (int j = 0; j < K::TN; ++j)
            if (n0 + j >= n) {
#pragma unroll
                for (int q = 0; q < K::TP; ++q) h[q][j] = make2((C)0, (C)0);
            }
    }
#pragma unroll
    for (int q = 0; q < K::TP; ++q) {
        if (MAIN) {
            y2[q] = mul2(c2[0], h[q][0]);
#pragma unroll
            for (int j = 1; j < K::TN; ++j) y2[q] = fma2(c2[j], h[q][j], y2[q]);
        } else {
            total[q] = add2(total[q], dt2[q]);
        }
    }
    if (MAIN) put<K::TP>(&sm.y[t][nl][d0], y2);
}

// MAIN: outputs.  Otherwise only what each segment leaves behind: its end state from a zero state, its sum of steps.
template <class K, bool MAIN>
__global__ void __launch_bounds__(SCAN_WARPS * 32) scan_kernel(const __grid_constant__ ScanArgs p)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, LN = K::LN, TD = K::TD, TN = K::TN, TP = K::TP;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanFwdSmem<K> &sm = reinterpret_cast<ScanFwdSmem<K> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place<K>(p, warp, w)) return;

    const int n = p.n, nl = lane / K::LD, d0 = (lane % K::LD) * TD, n0 = nl * TN, nd = w.nch - d0;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0 + d0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0 + d0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 + d0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    T *y = static_cast<T *>(p.y.p) + w.line * p.y.line + w.c0 + d0;
    const int64_t part = (int64_t)w.c0 * n, dn = p.d * n;
    const C *state = static_cast<const C *>(p.state);
    C *state_out = static_cast<C *>(p.state_out);

    // sequences without rows end as they began
    if (MAIN && state_out && p.rows.table && blockIdx.x == 0) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.table[2 * p.rows.live + 1 + e] * dn + part;
            for (int i = lane; i < w.nch * n; i += 32) state_out[at + i] = state ? state[at + i] : (C)0;
        }
    }
    if (w.r0 >= w.r1) return;

    V A2[TP][TN], h[TP][TN], total[TP], bias[TP], skip[TP];
    const bool plain = load_decay<K>(p.A, part, n, w.nch, lane, A2) && p.softplus;
    zero_part<K>(h);
#pragma unroll
    for (int q = 0; q < TP; ++q) {
        total[q] = make2((C)0, (C)0);
        bias[q] = pair_of<K>(p.dt_bias, w.c0 + d0, nd, q);
        skip[q] = pair_of<K>(MAIN ? p.D : nullptr, w.c0 + d0, nd, q);
    }

    int64_t k = p.rows.find(w.r0);
    if (MAIN && w.seg > 0 && p.rows.start(k) < w.r0) {
        // the state that the segments before this one leave: of the first that holds rows of this sequence, its end
        // state; each later one decays what came before by its own sum of steps
        scan_join<K>(p, w, (int)(p.rows.start(k) / p.seg_rows), w.seg, 1, lane, A2, h);
    }

    ScanLoad<K> xl, dl, zl;
    ScanLoadN<K, 32> bl, cl;
    auto fetch = [&](int64_t r) {
        xl.load(x, p.x.row, r, w.r1, nd, p.x.wide, nl);
        dl.load(dt, p.dt.row, r, w.r1, nd, p.dt.wide, nl);
        bl.load(B, p.B.row, r, w.r1, n, p.B.wide, lane);
        if (MAIN) cl.load(Cc, p.C.row, r, w.r1, n, p.C.wide, lane);
    };
    fetch(w.r0);

    for (int64_t rt = w.r0; rt < w.r1; rt += R) {
        // stage
#pragma unroll
        for (int i = 0; i < K::PER; ++i) {
            const int row = nl + LN * i;
            if (row >= R) break;
            V a[TP], b[TP];
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                a[q] = add2(make2(dl.v[i].get(2 * q), dl.v[i].get(2 * q + 1)), bias[q]);
                if (p.softplus) a[q] = softplus2(a[q]);
                b[q] = mul2(a[q], make2(xl.v[i].get(2 * q), xl.v[i].get(2 * q + 1)));
            }
            put<TP>(&sm.dt[row][d0], a);
            put<TP>(&sm.u[row][d0], b);
        }
        bl.stage(sm.b, lane);
        if (MAIN) cl.stage(sm.c, lane);
        const auto xc = xl;
        if (MAIN && z) zl.load(z, p.z.row, rt, w.r1, nd, p.z.wide, nl);
        if (rt + R < w.r1) fetch(rt + R);
        const uint32_t st = p.rows.starts(rt, R, k, lane);
        const int nr = (int)min((int64_t)R, w.r1 - rt);
        __syncwarp();
        if (MAIN && p.kept) {
            const int64_t tiles = (p.rows.rows + R - 1) / R;
            store_part<K>(static_cast<C *>(p.kept) + (w.line * tiles + rt / R) * dn + part, n, w.nch, lane, h);
        }
        for (int t = 0; t < nr;) {
            if ((st >> t) & 1u) {
                if (rt + t > p.rows.start(k)) ++k;
                if (state)
                    load_part<K>(state + p.rows.number(k, w.line) * dn + part, n, w.nch, lane, h);
                else
                    zero_part<K>(h);
            }
            const uint32_t later = st >> (t + 1);
            const int te = later ? min(nr, t + __ffs(later)) : nr;
            if (plain) {
                for (; t + 4 <= te; t += 4) {
                    scan_row<K, MAIN, true, 0>(sm, t, d0, n0, nl, n, A2, h, total);
                    scan_row<K, MAIN, true, 1>(sm, t + 1, d0, n0, nl, n, A2, h, total);
                    scan_row<K, MAIN, true, 2>(sm, t + 2, d0, n0, nl, n, A2, h, total);
                    scan_row<K, MAIN, true, 3>(sm, t + 3, d0, n0, nl, n, A2, h, total);
                }
            }
#pragma unroll 1
            for (; t < te; ++t) scan_row<K, MAIN, false, 0>(sm, t, d0, n0, nl, n, A2, h, total);
            if (MAIN && state_out && ((st >> t) & 1u))
                store_part<K>(state_out + p.rows.number(k, w.line) * dn + part, n, w.nch, lane, h);
        }
        __syncwarp();
        if (MAIN) {
#pragma unroll
            for (int i = 0; i < K::PER; ++i) {
                const int row = nl + LN * i;
                if (row >= nr) break;
                V v[TP];
                // each row's parts from another lane group on, so that rows read together lie on other banks
                get<TP>(&sm.y[row][nl][d0], v);
#pragma unroll
                for (int e = 1; e < LN; ++e) {
                    V o[TP];
                    get<TP>(&sm.y[row][(nl + e) % LN][d0], o);
#pragma unroll
                    for (int q = 0; q < TP; ++q) v[q] = add2(v[q], o[q]);
                }
                C out[TD];
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    v[q] = fma2(skip[q], make2(xc.v[i].get(2 * q), xc.v[i].get(2 * q + 1)), v[q]);
                    if (z) {
                        const V g = make2(zl.v[i].get(2 * q), zl.v[i].get(2 * q + 1));
                        v[q] = mul2(v[q], mul2(g, sigmoid2(g)));
                    }
                    out[2 * q] = v[q].x, out[2 * q + 1] = v[q].y;
                }
                Pack<T, TD> o;
                o.set(out);
                o.store(y + (rt + row) * p.y.row, nd, p.y.wide);
            }
            __syncwarp();
        }
    }
    if (!MAIN) scan_leave<K>(p, w, lane, h, total);
}

template <class K> cudaError_t scan_run(const ScanArgs &p, cudaStream_t s)
{
    const int64_t per = p.d / p.groups, tiles = (per + K::CW - 1) / K::CW;
    const int64_t gy = p.groups * ((tiles + SCAN_WARPS - 1) / SCAN_WARPS), gx = p.lines * p.segs;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    static_assert(scan_fwd_aligned<K>, "staged rows lie on 16 bytes");
    constexpr int bytes = SCAN_WARPS * (int)sizeof(ScanFwdSmem<K>);
    if (p.segs > 1) {
        cudaError_t e = cudaFuncSetAttribute(scan_kernel<K, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        scan_kernel<K, false><<<grid, SCAN_WARPS * 32, bytes, s>>>(p);
    }
    cudaError_t e = cudaFuncSetAttribute(scan_kernel<K, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_kernel<K, true><<<grid, SCAN_WARPS * 32, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
